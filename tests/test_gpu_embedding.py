"""Embedding lookup and its gradient by sorted tokens, against the float64 oracle.

A looked-up value is one fp32 product rounded to the table's type: 2^-24 + u of it.  A row of
the gradient is a sum of its k tokens in fp32, in any order: within (k + 3) 2^-24 of the sum of
the terms' sizes."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,v,d", [(1, 1, 1), (8, 50, 1024), (77, 1000, 131)])
def test_lookup(t, v, d, dt, idt):
    require_gpu()
    from bit_quantized_shampoo_amd import embedding
    rng = np.random.default_rng(t)
    table = torch.from_numpy(rng.standard_normal((v, d + 3)).astype(np.float32)).cuda().to(DT[dt])[:, 1:1 + d]
    ids = rng.integers(0, v, t)
    if t > 4:
        ids[[0, 2, 4]] = [-1, v, np.iinfo(np.int32).max]
    announce(f"embedding {t} of {v}x{d} {dt} {idt}")
    out = torch.full((t, d + 2), 9.0, dtype=DT[dt], device="cuda")
    embedding(table, torch.from_numpy(ids).to(idt).cuda(), scale=0.37, out=out[:, :d])
    ref = o.embedding(_np(table), ids, float(np.float32(0.37)))
    assert np.all(np.abs(_np(out[:, :d]) - ref) <= (2.0 ** -24 + U[dt]) * np.abs(ref) + (2.0 ** -25 if dt == "f16" else 0))
    assert bool((out[:, d:] == 9).all())


def _ids(rng, t, v, how):
    if how == "uniform":
        ids = rng.integers(0, v, t)
    elif how == "one":
        ids = np.full(t, v // 2)
    elif how == "few":
        ids = rng.choice([0, v // 3, v - 1], t)
    elif how == "none":
        ids = rng.choice([-1, v, -(1 << 31)], t)
    else:                                             # frequencies 1 / rank
        ids = np.minimum((np.exp(rng.random(t) * np.log(v + 1.0)) - 1).astype(np.int64), v - 1)
    if how not in ("one", "none") and t > 3:
        ids[rng.random(t) < 0.05] = -1
    return ids


def _check_grad(t, v, d, dt, how, accumulate, idt=torch.int64, pad=0, seed=0):
    from bit_quantized_shampoo_amd import embedding_grad
    rng = np.random.default_rng(seed + t)
    ids = _ids(rng, t, v, how)
    dout = torch.from_numpy(rng.standard_normal((t, d + pad)).astype(np.float32)).cuda().to(DT[dt])[:, :d]
    g0 = torch.from_numpy(rng.standard_normal((v, d + pad)).astype(np.float32)).cuda()
    if not accumulate:
        g0[:, :d] = float("nan")
    out = g0.clone()
    dev_ids = torch.from_numpy(ids).to(idt).cuda()
    announce(f"embedding grad T={t} V={v} D={d} {dt} {how} accumulate={accumulate} pad={pad}")
    embedding_grad(dout, dev_ids, v, scale=1.7, out=out[:, :d], accumulate=accumulate)
    torch.cuda.synchronize()
    # the oracle, one numpy call per array for the larger cases
    keep = (ids >= 0) & (ids < v)
    x = float(np.float32(1.7)) * _np(dout)
    ref, size, count = np.zeros((v, d)), np.zeros((v, d)), np.zeros(v)
    np.add.at(ref, ids[keep], x[keep])
    np.add.at(size, ids[keep], np.abs(x[keep]))
    np.add.at(count, ids[keep], 1)
    if t <= 40:
        assert np.allclose(ref, o.embedding_grad(_np(dout), ids, v, float(np.float32(1.7))), rtol=1e-12, atol=1e-300)
    if accumulate:
        ref, size = ref + _np(g0)[:, :d], size + np.abs(_np(g0)[:, :d])
    got = _np(out)[:, :d]
    assert np.all(np.abs(got - ref) <= (count[:, None] + 3) * 2.0 ** -24 * size)
    if accumulate:
        assert torch.equal(out[torch.from_numpy(count == 0).cuda()], g0[torch.from_numpy(count == 0).cuda()])
    assert torch.equal(torch.nan_to_num(out[:, d:]), torch.nan_to_num(g0[:, d:]))
    out2 = g0.clone()
    embedding_grad(dout, dev_ids, v, scale=1.7, out=out2[:, :d], accumulate=accumulate)
    assert torch.equal(out[:, :d], out2[:, :d])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("t,v,d,dt,how", [
    (0, 7, 5, "f32", "uniform"), (1, 1, 1, "f32", "uniform"), (1, 300, 64, "bf16", "uniform"),
    (15, 4, 9, "f16", "few"), (16, 5, 600, "f32", "one"), (17, 5, 600, "bf16", "one"), (40, 513, 33, "bf16", "zipf"),
    (1025, 700, 100, "f32", "zipf"), (3000, 70000, 24, "bf16", "uniform"), (2000, 3, 520, "f16", "few"),
    (777, 50, 8, "f32", "none"), (16384, 9, 8, "bf16", "one"),
])
def test_grad(t, v, d, dt, how, accumulate):
    require_gpu()
    _check_grad(t, v, d, dt, how, accumulate)


@pytest.mark.parametrize("t,v,d,dt,how,idt", [
    (2, 2, 3, "f32", "few", torch.int64), (31, 6, 8, "f32", "few", torch.int32), (33, 1 << 20, 2, "f32", "uniform", torch.int64),
    (1024, 30, 16, "bf16", "zipf", torch.int32), (4095, 900, 8, "f32", "zipf", torch.int64),
    (4096, 1, 8, "bf16", "one", torch.int32), (4096, 1 << 24, 1, "f32", "uniform", torch.int64),
    (4097, 900, 8, "f32", "zipf", torch.int32), (5000, 3, 24, "f16", "few", torch.int64),
    (8191, 5003, 16, "f32", "uniform", torch.int64), (16383, 70000, 8, "bf16", "zipf", torch.int32),
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_around_the_sorts_limits(t, v, d, dt, how, idt, accumulate):
    """Few tokens are placed by counting, more by digits in ranges of ids."""
    require_gpu()
    _check_grad(t, v, d, dt, how, accumulate, idt)


@pytest.mark.parametrize("t,v,d,dt,how,idt", [
    (16385, 511, 16, "f32", "zipf", torch.int32), (20000, 300000, 8, "bf16", "uniform", torch.int64),
    (40000, 65536, 8, "f32", "zipf", torch.int64), (30000, 2, 8, "f32", "few", torch.int32),
    (9000, 1 << 20, 8, "bf16", "uniform", torch.int32), (9000, 1 << 24, 1, "f32", "uniform", torch.int64),
])
def test_grad_sorted_in_blocks(t, v, d, dt, how, idt):
    """More tokens, or wider ids, than one workgroup's sort takes."""
    require_gpu()
    _check_grad(t, v, d, dt, how, False, idt)
    _check_grad(t, v, d, dt, how, True, idt, pad=3)


def test_grad_strided():
    require_gpu()
    _check_grad(500, 64, 77, "bf16", "zipf", False, torch.int32, pad=4)
    _check_grad(500, 64, 77, "f32", "zipf", True, torch.int64, pad=1)


def test_grad_is_the_difference_of_the_lookup():
    """<dout, embedding(E + h X) - embedding(E)> / h = <grad, X>: the lookup is linear, so float32
    roundings decide (1e-5 of the sum of the terms' sizes, for 2000 terms)."""
    require_gpu()
    from bit_quantized_shampoo_amd import embedding, embedding_grad
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(50, 40, generator=g, device="cuda")
    x = torch.randn(50, 40, generator=g, device="cuda")
    ids = torch.randint(-2, 52, (50,), generator=g, device="cuda")
    dout = torch.randn(50, 40, generator=g, device="cuda")
    announce("embedding differences")
    grad = embedding_grad(dout, ids, 50, scale=0.5).double()
    a = embedding(table + x, ids, scale=0.5).double() - embedding(table, ids, scale=0.5).double()
    left, right = (dout.double() * a).sum(), (grad * x.double()).sum()
    size = (dout.double() * a).abs().sum()
    assert float((left - right).abs()) <= 1e-5 * float(size)


def test_lookup_and_gradient_beyond_32_bit_offsets():
    require_gpu()
    from bit_quantized_shampoo_amd import embedding, embedding_grad
    v, d = 70000, 32768                               # 2.3e9 elements
    announce("embedding with 64-bit offsets")
    table = torch.zeros((v, d), dtype=torch.bfloat16, device="cuda")
    table[v - 1] = 2.0
    ids = torch.tensor([v - 1, 0, v - 1], device="cuda")
    out = embedding(table, ids, scale=1.5)
    assert bool((out[0] == 3).all()) and bool((out[1] == 0).all()) and bool((out[2] == 3).all())
    del table
    grad = embedding_grad(out, ids, v)
    assert bool((grad[v - 1] == 6).all()) and float(grad[v - 2].abs().sum()) == 0
    assert float(grad[: v - 1].abs().amax()) == 0


def test_captured_graphs():
    """Lookup and gradient (sorted at once, and in blocks) from captured graphs, replayed with
    other work between the replays, against the eager results."""
    require_gpu()
    from bit_quantized_shampoo_amd import embedding, embedding_grad
    gen = torch.Generator(device="cuda").manual_seed(9)
    for t, v in ((3000, 700), (20000, 5000)):
        table = torch.randn(v, 40, generator=gen, device="cuda").bfloat16()
        ids = torch.randint(-3, v + 3, (t,), generator=gen, device="cuda")
        call = lambda: (lambda o: (o, embedding_grad(o, ids, v, scale=0.5)))(embedding(table, ids, scale=2.0))  # noqa: E731
        want = call()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        announce(f"embedding graph {t} of {v}")
        with torch.cuda.stream(s):
            call()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = call()
        for _ in range(3):
            for x in got:
                x.zero_()
            torch.randn(1000, 1000, device="cuda").sum().item()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
