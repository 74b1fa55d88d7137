"""A stack of residual feed-forward blocks trained with every product in 8-bit floating point, on one GPU:

    embedding -> dropout -> norm -> [ gated feed-forward -> norm, dropout, gate, residual sum, next norm ] x layers
    -> logits

Forward and input-gradient products read weights quantised once a step, in both orientations; the norm
before a product writes its operand in 8 bits beside the result.  Weight gradients come from 8-bit
activation checkpoints, and the matrices take the 4-bit Shampoo step.  Dropout keeps no mask: the
backward pass draws the same numbers again.

The task is to learn a fixed rule that pairs every token with a word.

    python examples/residual_blocks.py [--steps N]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_shampoo_amd as s4  # noqa: E402


class Network:
    """float32 weights; activations of `dtype`."""

    def __init__(self, vocab=64, dim=64, hidden=160, layers=2, p=0.1, residual_scale=1.0, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.layers, self.p, self.rho, self.dtype = vocab, layers, p, residual_scale, dtype
        self.scale = math.sqrt(dim)

        def matrix(n, k):
            return torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)

        self.table = matrix(vocab, dim) / self.scale
        self.up = [[matrix(hidden, dim), matrix(hidden, dim), matrix(dim, hidden)] for _ in range(layers)]
        self.out = matrix(vocab, dim)
        # norms before each block and before the logits, norms and gates behind each block
        self.norm = [torch.ones(dim, device="cuda") for _ in range(layers + 1)]
        self.post = [torch.ones(dim, device="cuda") for _ in range(layers)]
        self.gate = [torch.full((dim,), 0.5, device="cuda") for _ in range(layers)]

    def matrices(self):
        return [self.table] + [w for block in self.up for w in block] + [self.out]

    def vectors(self):
        return self.norm + self.post + self.gate

    def forward(self, ids, seed=0, step=0, p=None):
        """Logits, and what backward needs.  Dropout draws by (seed, step)."""
        p = self.p if p is None else p
        calls = step * (self.layers + 1)
        w8 = [[s4.fp8_store_weight(w, transposed=True) for w in block] for block in self.up]
        out8 = s4.fp8_store_weight(self.out, transposed=True)
        x = s4.dropout(s4.embedding(self.table.to(self.dtype), ids, scale=self.scale), p, seed, calls)
        x, y, y8, stats = s4.block_norm_forward(x, self.norm[0], save8=True)
        saved = []
        for i in range(self.layers):
            drop = {"p": p, "seed": seed, "offset": calls + 1 + i}
            kept = {"x": x, "stats": stats, "y": s4.act8_store(y), "drop": drop}
            (wg, _), (wu, _), (wd, _) = w8[i]
            h, kept["gate"], kept["up"], kept["h"] = s4.activation_forward(s4.fp8_linear(y8, wg, dtype=self.dtype),
                                                                           s4.fp8_linear(y8, wu, dtype=self.dtype))
            kept["d"] = s4.fp8_linear(h, wd)
            x, y, y8, stats = s4.block_norm_forward(x, self.norm[i + 1], kept["d"], post_weight=self.post[i],
                                                    gate=self.gate[i], residual_scale=self.rho, save8=True, **drop)
            saved.append(kept)
        logits = s4.fp8_linear(y8, out8[0], dtype=self.dtype)
        return logits, (ids, seed, calls, p, w8, out8, saved, x, stats, s4.act8_store(y))

    def backward(self, dlogits, state):
        """float32 gradients of matrices() and of vectors()."""
        ids, seed, calls, p, w8, out8, saved, x, stats, y = state
        matrices, norms, posts, gates = [], [None] * (self.layers + 1), [], []
        grad_out = s4.act8_weight_grad(dlogits, y)
        dy, dres = s4.fp8_linear(dlogits, out8[1]), None
        for i in reversed(range(self.layers)):
            k = saved[i]
            dres, dd, norms[i + 1], post, gate = s4.block_norm_backward(dy, dres, x, self.norm[i + 1], stats, h=k["d"],
                                                                        post_weight=self.post[i], gate=self.gate[i],
                                                                        residual_scale=self.rho, **k["drop"])
            (_, wg), (_, wu), (_, wd) = w8[i]
            dgate, dup = s4.activation_backward(s4.fp8_linear(dd, wd), k["gate"], k["up"])
            matrices[:0] = [s4.act8_weight_grad(dgate, k["y"]), s4.act8_weight_grad(dup, k["y"]), s4.act8_weight_grad(dd, k["h"])]
            posts.insert(0, post)
            gates.insert(0, gate)
            dy = s4.fp8_linear(dgate, wg)
            s4.fp8_linear(dup, wu, out=dy, accumulate=True)
            x, stats = k["x"], k["stats"]
        dx, _, norms[0], _, _ = s4.block_norm_backward(dy, dres, x, self.norm[0], stats)
        dx = s4.dropout(dx, p, seed, calls, out=dx)
        table = s4.embedding_grad(dx, ids, self.vocab, scale=self.scale)
        return [table] + matrices + [grad_out], norms + posts + gates


def gradients(net, ids, targets, seed=0, step=0):
    """The mean log-probability's negative, and its gradients.  With the old log-probabilities being the
    present ones and advantages of 1, the policy loss's gradient is the likelihood's."""
    logits, state = net.forward(ids, seed, step)
    old = s4.token_logprobs(logits, targets)
    ones = torch.ones_like(old)
    _, logp, dlogits = s4.policy_loss(logits, targets, old, ones, ones / len(ids), dlogits=logits)
    return -logp.mean(), *net.backward(dlogits, state)


def train(steps=60, tokens=1024, lr=3e-3, seed=0, log=None):
    net = Network(seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    rule = torch.randperm(net.vocab, generator=gen, device="cuda")
    matrices = net.matrices()
    optimizer = s4.Shampoo4Blocks([tuple(w.shape) for w in matrices], s4.Shampoo4Config(root_cache=True))
    moments = [(torch.zeros_like(w), torch.zeros_like(w)) for w in matrices]
    losses = []
    for step in range(steps):
        ids = torch.randint(0, net.vocab, (tokens,), generator=gen, device="cuda")
        loss, grads, vectors = gradients(net, ids, rule[ids], seed, step)
        directions = optimizer.step(grads, step + 1, root_interval=2)
        optimizer.graft(grads, directions, matrices, moments, mode="adam", step=step + 1, lr=lr)
        for v, g in zip(net.vectors(), vectors):
            v -= lr * g
        losses.append(float(loss))
        if not math.isfinite(losses[-1]):
            raise RuntimeError(f"the loss is not finite at step {step}")
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
    if optimizer.check():
        raise RuntimeError("the optimizer saw a value that is not finite")
    optimizer.close()
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps, log=print)
