"""The residual block's operators together, as the example trains with them: its gradients against the same
network in float64, the same bits from a repeated and from a captured pass, and that it runs.

The float64 network quantises at the same places, by the definitions, and takes gradients of the
quantised products by the formulas.  The float32 run differs from it by roundings of about 1e-6, which move a
value over a border of its 8-bit format (spacing at least 2^-4 of it, 2^-8 of the block's largest for
checkpoints) for at most 2 * 1e-6 * 2^4 = 3.2e-5 of the elements, by at most 2^-3 of their size: 7e-4 of a
matrix's norm for each quantisation, of which 8 in the forward pass and 12 in the backward pass lie behind a
gradient: 1.4e-2."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def _module():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import residual_blocks
    return residual_blocks


def _q(x, rows=1):
    return o.fp8_load(*o.fp8_store(x, rows), x.shape[1], rows)


def _c(x):
    return o.act8_load(*o.act8_store(x), *x.shape)


def _oracle(net, ids, targets, seed, step):
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    t, dim, calls, eps = len(ids), net.table.shape[1], step * (net.layers + 1), float(np.float32(1e-6))
    p = np.float32(net.p)
    drop = [o.dropout_keep(t, dim, p, seed, calls + i) * o.dropout_scale(p) for i in range(net.layers + 1)]
    x = drop[0] * o.embedding(n(net.table), ids, net.scale)
    y = x * o.rstd(x, eps) * n(net.norm[0])
    w8 = [[_q(n(w), 128) for w in block] for block in net.up]
    out8 = _q(n(net.out), 128)
    saved, xs = [], [x]
    for i in range(net.layers):
        wg, wu, wd = w8[i]
        a, b = _q(y) @ wg.T, _q(y) @ wu.T
        h = o.activation(a, "silu") * b
        d = _q(h) @ wd.T
        saved.append((_c(y), _c(a), _c(b), _c(h), d))
        x = o.block_end(x, d, n(net.post[i]), n(net.gate[i]), drop[i + 1], net.rho, eps)
        xs.append(x)
        y = x * o.rstd(x, eps) * n(net.norm[i + 1])
    z = _q(y) @ out8.T
    lp = o.log_softmax(z)
    loss = -lp[np.arange(t), targets].mean()
    dz = np.exp(lp)
    dz[np.arange(t), targets] -= 1
    dz /= t
    matrices, norms, posts, gates = [dz.T @ _c(y)], [None] * (net.layers + 1), [], []
    dy, dres = _q(dz) @ _q(n(net.out).T, 128).T, None
    for i in reversed(range(net.layers)):
        y8, a8, b8, h8, d = saved[i]
        g, _ = o.block_backward(dy, dres, xs[i + 1], n(net.norm[i + 1]), d, n(net.post[i]), n(net.gate[i]), drop[i + 1],
                                net.rho, eps)
        norms[i + 1], dres = g["dweight"], g["dx"]
        posts.insert(0, g["dpost"])
        gates.insert(0, g["dgate"].sum(0))
        wg, wu, wd = (_q(n(w).T, 128) for w in net.up[i])
        dh = _q(g["dh"]) @ wd.T
        da, db = dh * b8 * o.activation_derivative(a8, "silu"), dh * o.activation(a8, "silu")
        matrices[:0] = [da.T @ y8, db.T @ y8, g["dh"].T @ h8]
        dy = _q(da) @ wg.T + _q(db) @ wu.T
    g, _ = o.block_backward(dy, dres, xs[0], n(net.norm[0]), None, None, None, None, 1.0, eps)
    norms[0] = g["dweight"]
    return loss, [o.embedding_grad(drop[0] * g["dx"], ids, net.vocab, net.scale)] + matrices, norms + posts + gates


def test_gradients_of_the_whole():
    require_gpu()
    m = _module()
    net = m.Network(vocab=50, dim=72, hidden=200, layers=2, p=0.2, residual_scale=0.8, dtype=torch.float32, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for v in net.vectors():
        v += 0.1 * torch.randn(v.shape, generator=g, device="cuda")
    ids = torch.randint(0, 50, (130,), generator=g, device="cuda")
    targets = torch.randint(0, 50, (130,), generator=g, device="cuda")
    announce("residual blocks, gradients")
    loss, matrices, vectors = m.gradients(net, ids, targets, seed=11, step=2)
    want = _oracle(net, ids.cpu().numpy(), targets.cpu().numpy(), 11, 2)
    assert abs(float(loss) - want[0]) <= 1.4e-2 * want[0]
    for i, (a, b) in enumerate(zip(matrices + vectors, want[1] + want[2])):
        a = a.double().cpu().numpy()
        assert a.shape == b.shape
        assert np.linalg.norm(a - b) <= 1.4e-2 * np.linalg.norm(b), i


def test_repeated_and_captured_passes():
    require_gpu()
    m = _module()
    net = m.Network(vocab=60, dim=136, hidden=300, layers=2, p=0.1, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    ids, targets = (torch.randint(0, 60, (200,), generator=g, device="cuda") for _ in range(2))

    def call():
        loss, matrices, vectors = m.gradients(net, ids, targets, seed=1, step=7)
        return [loss] + matrices + vectors

    announce("residual blocks, repeated and captured")
    want = call()
    assert all(torch.equal(a, b) for a, b in zip(want, call()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = call()
    for _ in range(3):
        for x in got[1:]:
            x.zero_()
        torch.randn(1000, 1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[1:], got[1:]))


def test_example_runs():
    require_gpu()
    announce("example residual blocks, 4 steps")
    losses = _module().train(steps=4, tokens=256)
    assert len(losses) == 4 and all(np.isfinite(losses))
