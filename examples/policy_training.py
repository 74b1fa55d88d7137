"""Policy training of a small language model with the library's training operators and the
4-bit Shampoo step, end to end on one GPU:

    embedding -> gated feed-forward blocks -> logits -> clipped policy loss with a KL term,

backward from 8-bit activation checkpoints, every weight gradient straight into the step.
Plain matrix products (y = x W^T and dx = dy W) are torch's.

The task is a contextual bandit: for every token the model picks a word and is rewarded when
it is the one that a fixed rule pairs with the token.

    python examples/policy_training.py [--steps N]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_shampoo_amd as s4  # noqa: E402
from bit_quantized_shampoo_amd.blocking import block_diagonal_sides, block_shapes, block_views, plan_blocks  # noqa: E402


class Model:
    """float32 weights, bfloat16 activations; what the backward pass needs is kept in 8 bits."""

    def __init__(self, vocab=64, dim=64, hidden=192, layers=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.layers, self.scale = vocab, layers, math.sqrt(dim)
        shapes = [(vocab, dim)] + [(hidden, dim), (hidden, dim), (dim, hidden)] * layers + [(vocab, dim)]
        self.weights = [torch.randn(s, generator=g, device="cuda") / math.sqrt(s[1]) for s in shapes]
        self.weights[0] /= self.scale

    def forward(self, ids, weights=None, keep=True):
        """Logits, and what backward needs (None with keep=False)."""
        w = [x.bfloat16() for x in (self.weights if weights is None else weights)]
        x = s4.embedding(w[0], ids, scale=self.scale)
        saved = []
        for i in range(self.layers):
            wg, wu, wd = w[1 + 3 * i:4 + 3 * i]
            x8 = s4.act8_store(x) if keep else None
            h, g8, u8, h8 = s4.activation_forward(x @ wg.t(), x @ wu.t(), kind="silu", checkpoint=keep, save_output=keep)
            x = x + h @ wd.t()
            saved.append((x8, g8, u8, h8))
        logits = x @ w[-1].t()
        return logits, (w, saved, s4.act8_store(x)) if keep else None

    def backward(self, dlogits, ids, state):
        """float32 gradients of every weight, in the order of `weights`."""
        w, saved, x8 = state
        grads = [None] * len(w)
        grads[-1] = s4.act8_weight_grad(dlogits, x8)
        dx = dlogits @ w[-1]
        for i in reversed(range(self.layers)):
            wg, wu, wd = w[1 + 3 * i:4 + 3 * i]
            x8, g8, u8, h8 = saved[i]
            grads[3 + 3 * i] = s4.act8_weight_grad(dx, h8)
            dgate, dup = s4.activation_backward(dx @ wd, g8, u8, kind="silu")
            grads[1 + 3 * i] = s4.act8_weight_grad(dgate, x8)
            grads[2 + 3 * i] = s4.act8_weight_grad(dup, x8)
            dx = dx + dgate @ wg + dup @ wu
        grads[0] = s4.embedding_grad(dx, ids, self.vocab, scale=self.scale)
        return grads


def train(steps=60, tokens=2048, inner=2, lr=3e-3, seed=0, log=None):
    """Mean reward of every step."""
    model = Model(seed=seed)
    reference = [w.clone() for w in model.weights]
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    rule = torch.randperm(model.vocab, generator=gen, device="cuda")
    # the tables' long side keeps a diagonal factor, as it would at a real vocabulary's size
    plans = plan_blocks([tuple(w.shape) for w in model.weights], block=None, max_dim=192)
    optimizer = s4.Shampoo4Blocks(block_shapes(plans), s4.Shampoo4Config(root_cache=True),
                                  diagonal=block_diagonal_sides(plans))
    blocks = block_views(model.weights, plans)
    moments = [(torch.zeros_like(b), torch.zeros_like(b)) for b in blocks]
    rewards, t = [], 0
    for step in range(steps):
        ids = torch.randint(0, model.vocab, (tokens,), generator=gen, device="cuda")
        with_prompt = torch.rand(tokens, generator=gen, device="cuda") < 0.1       # tokens that are not answers
        logits, _ = model.forward(ids, keep=False)
        # a sample of softmax(logits): the largest of logits plus Gumbel noise
        noise = torch.rand(logits.shape, generator=gen, device="cuda").clamp_(1e-20, 1 - 1e-7)
        actions = (logits.float() - torch.log(-torch.log(noise))).argmax(1)
        reward = (actions == rule[ids]).float()
        old = s4.token_logprobs(logits, actions)
        ref = s4.token_logprobs(model.forward(ids, reference, keep=False)[0], actions)
        advantage = (reward - reward.mean()) / (reward.std() + 1e-4)
        weight = (~with_prompt).float()
        weight /= weight.sum()
        for _ in range(inner):
            t += 1
            logits, state = model.forward(ids)
            loss, _, dlogits = s4.policy_loss(logits, actions, old, advantage, weight, ref_logp=ref, clip_low=0.2,
                                              clip_high=0.28, kl_coef=1e-3, dlogits=logits)
            grads = block_views(model.backward(dlogits, ids, state), plans)
            directions = optimizer.step(grads, t, root_interval=2)
            optimizer.graft(grads, directions, blocks, moments, mode="adam", step=t, lr=lr)
        if not math.isfinite(float(loss)):
            raise RuntimeError(f"the loss is not finite at step {step}")
        rewards.append(float(reward.mean()))
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  reward {rewards[-1]:.3f}  loss {float(loss):+.4f}")
    if optimizer.check():
        raise RuntimeError("the optimizer saw a value that is not finite")
    optimizer.close()
    return rewards


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps, log=print)
