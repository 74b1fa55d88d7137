"""The ends of a residual block and dropout, on the GPU against the float64 oracle.

Tolerances, with u the stored type's unit roundoff and e = 2^-24:
* which elements are dropped is exact; a kept one is one fp32 product, rounded: e + u;
* rstd: a sum of squares of at most 16 terms in a lane, 6 steps across lanes and 16 waves (38 e, halved by
  the root), a division, an addition, a root and a division: 32 e covers it;
* x' = rho x + gate z: 38 e of |gate z|, 2 e of |rho x|, then u;  y of the x' that was stored: 36 e, then u;
* dx: terms with up to three factors of rstd (96 e), the mean of t xh (38 e of the mean of sizes) and eight
  operations: 160 e of the oracle's sizes, then u;  dgate, another 40 e;  dh: the same again for its own
  row sum, 320 e;
* sums over rows: a row's terms (40, 240 and 200 e) and one rounding for each of T rows: (T + those) e
  of the sum of sizes."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -140, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
E = 2.0 ** -24
SEED, OFFSET = 0x123456789ABCDEF0, (5 << 32) + 7


def _np(t):
    return t.detach().double().cpu().numpy()


def _rand(rng, t, c, dt, scale=1.0):
    x = scale * rng.standard_normal((t, c)) * np.exp(0.5 * rng.standard_normal((1, c)))
    return torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dt])


def _vec(rng, c, mean):
    return torch.from_numpy((mean + 0.2 * rng.standard_normal(c)).astype(np.float32)).cuda()


def _strided(x, pad, offset=0):
    t, c = x.shape
    big = torch.full((t, c + pad + offset), float("nan"), dtype=x.dtype, device=x.device)
    big[:, offset:offset + c] = x
    return big[:, offset:offset + c]


def _close(got, ref, tol, what):
    bad = ~(np.abs(_np(got) - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(np.abs(_np(got) - ref) / tol)))


# -- dropout -------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,c,p", [(1, 1, 0.5), (3, 7, 0.3), (4, 512, 0.1), (9, 600, 0.9), (2, 1025, 0.02), (5, 40, 0.0)])
def test_dropout(t, c, p, dt):
    require_gpu()
    from bit_quantized_shampoo_amd import dropout
    rng = np.random.default_rng(t + c)
    x = _strided(_rand(rng, t, c, dt), 3, 1)
    announce(f"dropout {t}x{c} {dt} p={p}")
    y = dropout(x, p, SEED, OFFSET)
    keep = o.dropout_keep(t, c, np.float32(p), SEED, OFFSET)
    ref = np.where(keep, _np(x) * o.dropout_scale(np.float32(p)), 0.0)
    _close(y, ref, (2 * E + U[dt]) * np.abs(ref) + (TINY[dt] if p else 0), "dropout")
    assert torch.equal(y == 0, torch.from_numpy(~keep).cuda() | (x == 0))
    # the counter is added; the generator's state is the caller's
    counter = torch.tensor([3], dtype=torch.int64, device="cuda")
    assert torch.equal(dropout(x, p, SEED, OFFSET - 3, counter=counter), y)
    assert torch.equal(dropout(x, p, SEED - (1 << 64), OFFSET), y)                    # the seed modulo 2^64
    # in place, and what lies beside the rows
    out = torch.full((t, c + 5), 9.0, dtype=DT[dt], device="cuda")
    out[:, 2:2 + c] = x
    dropout(out[:, 2:2 + c], p, SEED, OFFSET, out=out[:, 2:2 + c])
    assert torch.equal(out[:, 2:2 + c], y) and bool((out[:, :2] == 9).all()) and bool((out[:, 2 + c:] == 9).all())


def test_dropout_of_values_that_are_not_finite():
    """A dropped infinity or NaN is 0; p in steps of 2^-16, down to nothing."""
    require_gpu()
    from bit_quantized_shampoo_amd import dropout
    keep = torch.from_numpy(o.dropout_keep(8, 100, 0.5, 1, 2)).cuda()
    announce("dropout of infinities and NaN")
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = torch.full((8, 100), bad, device="cuda").bfloat16()
        y = dropout(x, 0.5, 1, 2)
        assert bool((y[~keep] == 0).all()) and not bool(torch.isfinite(y[keep]).any())
    x = torch.randn(8, 100, device="cuda")
    assert torch.equal(dropout(x, 2.0 ** -18, 1, 2), x)
    most = dropout(x, 1 - 2.0 ** -16, 1, 2)
    assert torch.equal(most != 0, torch.from_numpy(o.dropout_keep(8, 100, 1 - 2.0 ** -16, 1, 2)).cuda())


def test_dropout_far_rows():
    """Row numbers beyond 16 bits and offsets beyond 32."""
    require_gpu()
    from bit_quantized_shampoo_amd import dropout
    t, c = 70001, 33000
    announce("dropout with 64-bit offsets")
    x = torch.ones((t, c), dtype=torch.bfloat16, device="cuda")
    dropout(x, 0.25, SEED, OFFSET, out=x)
    for row, col in ((0, 0), (65536, 512), (70000, 32992)):
        keep = o.dropout_keep(1, 8, 0.25, SEED, OFFSET, row0=row, col0=col)[0]
        assert np.array_equal(_np(x[row, col:col + 8]) != 0, keep)
    share = float((x != 0).float().mean())
    assert abs(share - 0.75) < 5 * np.sqrt(0.75 * 0.25 / (t * c)) + 2.0 ** -24


# -- the block ------------------------------------------------------------------------------

def _case(t, c, dt, post, gate, weight, p, rho, seed=0, scale=1.0):
    rng = np.random.default_rng(seed + 7 * t + c)
    v = {"x": _rand(rng, t, c, dt, 2.0 * scale), "h": _rand(rng, t, c, dt, scale), "dres": _rand(rng, t, c, dt, 1e-2)}
    v["post"] = _vec(rng, c, 0.5) if post else None
    v["gate"] = None if gate is None else _vec(rng, c, 0.6) if gate == "channel" else _rand(rng, t, c, dt, 0.5)
    v["weight"] = _vec(rng, c, 1.0) if weight else None
    v["dy"] = _rand(rng, t, c, dt, 1e-2) if weight else None
    v["drop"] = o.dropout_keep(t, c, np.float32(p), SEED, OFFSET) * o.dropout_scale(np.float32(p)) if p else None
    return v


def _check(t, c, dt, post, gate, weight, p, rho, strided=False, dres=True, eps=1e-5, scale=1.0):
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward, fp8_store
    v = _case(t, c, dt, post, gate, weight, p, rho, scale=scale)
    if strided:
        for k in ("x", "h", "dres", "dy"):
            v[k] = None if v[k] is None else _strided(v[k], 3, 1)
        if gate == "token":
            v["gate"] = _strided(v["gate"], 2)
    if not dres and weight:
        v["dres"] = None
    n = {k: None if a is None else a if isinstance(a, np.ndarray) else _np(a) for k, a in v.items()}
    kw = dict(post_weight=v["post"], gate=v["gate"], residual_scale=rho, eps=eps, p=p, seed=SEED, offset=OFFSET)
    announce(f"block {t}x{c} {dt} post={post} gate={gate} weight={weight} p={p} rho={rho} strided={strided} scale={scale}")
    x, y, y8, stats = block_norm_forward(v["x"], v["weight"], v["h"], save8=weight, **kw)
    rho = float(np.float32(rho))
    eps = float(np.float32(eps))
    z = o.block_end(np.zeros((t, c)), n["h"], n["post"], n["gate"], n["drop"], rho, eps)
    ref = rho * n["x"] + z
    _close(x, ref, 38 * E * np.abs(z) + 2 * E * np.abs(rho * n["x"]) + U[dt] * np.abs(ref) + TINY[dt], "x'")
    stored = _np(x)
    if post:
        r = o.rstd(n["h"], eps)
        _close(stats[0], r[:, 0], 32 * E * r[:, 0] + 2.0 ** -149, "h_rstd")
    if weight:
        r = o.rstd(stored, eps)
        _close(stats[1], r[:, 0], 32 * E * r[:, 0] + 2.0 ** -149, "rstd")
        ref = stored * r * n["weight"]
        _close(y, ref, (36 * E + U[dt]) * np.abs(ref) + TINY[dt], "y")
        want = fp8_store(y)
        assert torch.equal(y8.scales, want.scales)
        assert torch.equal(y8.codes.view(torch.uint8), want.codes.view(torch.uint8))
    else:
        assert y is None and y8 is None
    got = block_norm_backward(v["dy"], v["dres"], x, v["weight"], stats, h=v["h"], **kw)
    ref, size = o.block_backward(n["dy"], n["dres"], stored, n["weight"], n["h"], n["post"], n["gate"], n["drop"], rho, eps)
    bounds = {"dx": 160, "dh": 320, "dweight": t + 40, "dpost": t + 240, "dgate": 200}
    if gate == "channel":
        ref["dgate"], size["dgate"], bounds["dgate"] = ref["dgate"].sum(0), size["dgate"].sum(0), t + 200
    for name, a in zip(("dx", "dh", "dweight", "dpost", "dgate"), got):
        if (name == "dweight" and not weight) or (name == "dpost" and not post) or (name == "dgate" and gate is None):
            assert a is None
            continue
        u = U[dt] if a.dtype != torch.float32 else E
        _close(a, ref[name], bounds[name] * E * size[name] * (1 + u) + u * np.abs(ref[name]) + TINY[dt], name)
    again = block_norm_backward(v["dy"], v["dres"], x, v["weight"], stats, h=v["h"], **kw)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, again))
    return v, kw, (x, y, stats), got


OPTIONS = [(True, "channel", True, 0.1, 1.0), (False, "token", True, 0.0, 0.7071), (True, None, True, 0.0, 1.0),
           (False, None, True, 0.3, 0.5), (True, "token", False, 0.2, 1.0), (False, "channel", False, 0.0, 1.0)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,c", [(1, 1), (5, 7), (4, 64), (3, 129), (9, 513), (6, 1024), (5, 1030), (7, 2309), (2, 4096),
                                 (3, 4099), (2, 8192), (2, 8200), (2, 16384)])
def test_block_matches_oracle(t, c, dt):
    require_gpu()
    k = {"bf16": 0, "f16": 2, "f32": 4}[dt] + t
    for i in range(3 if c < 4096 else 1):
        _check(t, c, dt, *OPTIONS[(k + 2 * i) % 6], strided=(k + i) % 2 == 1, dres=(k + i) % 3 != 2)


@pytest.mark.parametrize("options", OPTIONS)
def test_block_options(options):
    require_gpu()
    for dt in DT:
        _check(11, 300, dt, *options, strided=True)
        _check(11, 1200, dt, *options)


def test_block_many_rows():
    """More rows than workgroups keep sums of at once."""
    require_gpu()
    _check(2100, 24, "f32", *OPTIONS[0])
    _check(2049, 7, "bf16", *OPTIONS[1])
    _check(1030, 1032, "bf16", *OPTIONS[0])


@pytest.mark.parametrize("t,c,dt,k", [(1, 8193, "f32", 1), (5, 12288, "f16", 5), (4, 12289, "bf16", 4), (3, 16383, "f32", 3),
                                      (520, 8200, "bf16", 0), (300, 9001, "f32", 2), (140, 16384, "bf16", 1)])
def test_block_wide_rows(t, c, dt, k):
    """Rows that the backward pass takes by ranges of columns, their two sums before; more rows than groups."""
    require_gpu()
    _check(t, c, dt, *OPTIONS[k], strided=t == 4, dres=t != 5)


def test_block_wide_rows_in_place():
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward
    for dt in ("bf16", "f32"):
        v, kw, (x, _, stats), got = _check(6, 10240, dt, True, "channel", True, 0.1, 0.5)
        announce(f"wide rows in place {dt}")
        h, dy, dres = v["h"].clone(), v["dy"].clone(), v["dres"].clone()
        out = block_norm_backward(dy, dres, x, v["weight"], stats, h=h, dx=dres, dh=h, **kw)
        assert out[0] is dres and out[1] is h
        assert all(torch.equal(a, b) for a, b in zip(out, got))
        dres = v["dres"].clone()
        out = block_norm_backward(dy, dres, x, v["weight"], stats, h=v["h"], dx=dy, dh=dres, **kw)
        assert all(torch.equal(a, b) for a, b in zip(out, got))


def test_block_rows_beyond_fp32_squares():
    """Rows whose squares leave fp32, and rows of very small values."""
    require_gpu()
    for scale in (1e25, 1e30, 1e-25):
        _check(6, 700, "f32", True, None, True, 0.0, 1.0, scale=scale, eps=1e-30 if scale < 1 else 1e-5)
        _check(3, 2100, "bf16", True, None, True, 0.0, 1.0, scale=scale)


def test_norm_alone():
    """Without a block: the first norm, forward and backward, and its gradient against differences."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward
    rng = np.random.default_rng(3)
    for dt, t, c in (("bf16", 5, 1024), ("f32", 4, 77), ("f16", 1, 3000)):
        x, w, dy, dres = _rand(rng, t, c, dt), _vec(rng, c, 1.0), _rand(rng, t, c, dt), _rand(rng, t, c, dt)
        announce(f"norm alone {t}x{c} {dt}")
        same, y, y8, stats = block_norm_forward(x, w, eps=1e-5)
        assert same is x and y8 is None
        eps = float(np.float32(1e-5))
        ref = _np(x) * o.rstd(_np(x), eps) * _np(w)
        _close(y, ref, (36 * E + U[dt]) * np.abs(ref) + TINY[dt], "y")
        dx, dh, dw, dp, dg = block_norm_backward(dy, dres, x, w, stats, eps=1e-5)
        assert dh is None and dp is None and dg is None
        ref, size = o.block_backward(_np(dy), _np(dres), _np(x), _np(w), None, None, None, None, 1.0, eps)
        _close(dx, ref["dx"], 160 * E * size["dx"] * (1 + U[dt]) + U[dt] * np.abs(ref["dx"]) + TINY[dt], "dx")
        _close(dw, ref["dweight"], (t + 41) * E * size["dweight"], "dweight")


def test_gradients_are_differences():
    """dx, dh and the vectors' gradients against a central difference of the float64 formulas along one direction
    each: fp32's roundings decide (320 e of the sum of sizes); the difference's own error is about 1e-9 of it."""
    require_gpu()
    v, kw, (x, _, _), got = _check(6, 90, "f32", True, "channel", True, 0.25, 0.7)
    n = {k: a if isinstance(a, np.ndarray) else _np(a) for k, a in v.items()}
    eps, rho = float(np.float32(1e-5)), float(np.float32(0.7))

    def loss(m):
        xx = o.block_end(m["x"], m["h"], m["post"], m["gate"], m["drop"], rho, eps)
        return np.sum(m["dres"] * xx) + np.sum(m["dy"] * xx * o.rstd(xx, eps) * m["weight"])

    rng = np.random.default_rng(6)
    for name, g in (("x", got[0]), ("h", got[1]), ("weight", got[2]), ("post", got[3]), ("gate", got[4])):
        d = rng.standard_normal(n[name].shape)
        h = 1e-5
        diff = (loss({**n, name: n[name] + h * d}) - loss({**n, name: n[name] - h * d})) / (2 * h)
        size = np.sum(np.abs(d) * np.abs(_np(g)))
        # x' is rounded before its norm (2^-24 of it), which the formula's x' is not: another 8 e
        assert abs(np.sum(d * _np(g)) - diff) <= 400 * E * size + 1e-7 * size, name


def test_in_place_and_aliases():
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward
    for dt, c in (("bf16", 600), ("f32", 2309)):
        v, kw, (x, y, stats), got = _check(5, c, dt, True, "channel", True, 0.1, 0.5)
        announce(f"block in place {dt} {c}")
        for target in ("x", "h"):
            a = {k: v[k].clone() for k in ("x", "h")}
            x2, y2, _, s2 = block_norm_forward(a["x"], v["weight"], a["h"], out=a[target], **kw)
            assert x2 is a[target] and torch.equal(x2, x) and torch.equal(y2, y) and torch.equal(s2, stats)
        h = v["h"].clone()
        x2, y2, _, _ = block_norm_forward(v["x"], v["weight"], h, y=h, **kw)
        assert torch.equal(x2, x) and torch.equal(h, y)
        for tx, th in (("dres", "h"), ("dy", "dres"), ("dres", "dy")):
            a = {k: v[k].clone() for k in ("dy", "dres", "h")}
            again = block_norm_backward(a["dy"], a["dres"], x, v["weight"], stats, h=a["h"], dx=a[tx], dh=a[th], **kw)
            assert all(torch.equal(p, q) for p, q in zip(got, again))


def test_rows_behind_and_padding_stay():
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_forward
    v, kw, (x, y, _), _ = _check(3, 77, "bf16", False, "token", True, 0.2, 1.0)
    big = [torch.full((6, 90), 4.0, device="cuda").bfloat16() for _ in range(2)]
    announce("block rows behind")
    block_norm_forward(v["x"], v["weight"], v["h"], out=big[0][:3, 1:78], y=big[1][:3, :77], **kw)
    assert torch.equal(big[0][:3, 1:78], x) and torch.equal(big[1][:3, :77], y)
    assert bool((big[0][3:] == 4).all()) and bool((big[0][:, :1] == 4).all()) and bool((big[0][:, 78:] == 4).all())
    assert bool((big[1][3:] == 4).all()) and bool((big[1][:, 77:] == 4).all())


def test_dropped_values_reach_nothing():
    """Without a norm behind the block, what is dropped may be infinite or NaN."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward
    v = _case(6, 200, "f32", False, "channel", True, 0.4, 1.0)
    kw = dict(gate=v["gate"], p=0.4, seed=SEED, offset=OFFSET)
    h2 = v["h"].clone()
    h2[torch.from_numpy(v["drop"] == 0).cuda()] = float("nan")
    announce("block with dropped NaN")
    a, b = (block_norm_forward(v["x"], v["weight"], h, **kw) for h in (v["h"], h2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (block_norm_backward(v["dy"], v["dres"], a[0], v["weight"], a[3], h=h, **kw) for h in (v["h"], h2))
    assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(ga, gb))


def test_no_rows():
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward, dropout
    announce("block without rows")
    e, w = torch.empty(0, 33, device="cuda"), torch.ones(33, device="cuda")
    assert dropout(e, 0.5, 1).shape == (0, 33)
    x, y, y8, stats = block_norm_forward(e, w, e, post_weight=w, gate=w, residual_scale=0.5, save8=True)
    assert x.shape == y.shape == (0, 33)
    dx, dh, dw, dp, dg = block_norm_backward(e, e, x, w, stats, h=e, post_weight=w, gate=w, residual_scale=0.5)
    assert dx.shape == dh.shape == (0, 33) and not bool(dw.any()) and not bool(dp.any()) and not bool(dg.any())


def test_binding_refusals():
    require_gpu()
    from bit_quantized_shampoo_amd import Shampoo4Error, block_norm_backward, block_norm_forward, dropout
    x, w, s = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda"), torch.zeros(2, 4, device="cuda")
    for f in (lambda: block_norm_forward(x), lambda: block_norm_forward(x, w, gate=w), lambda: block_norm_forward(x, w[:7]),
              lambda: block_norm_forward(x, w, residual_scale=2.0), lambda: block_norm_forward(x, None, x, save8=True),
              lambda: block_norm_forward(x, w, x[:3]), lambda: block_norm_forward(x, w, x, gate=x[:3]),
              lambda: block_norm_backward(None, x, x, w, s), lambda: block_norm_backward(x, x, x, None, s),
              lambda: block_norm_backward(None, None, x, None, s), lambda: block_norm_backward(x, x, x, w, s[:, :3]),
              lambda: block_norm_backward(x, x, x, w, s, gate=w), lambda: dropout(x, 0.5, 1, counter=s.long())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: block_norm_forward(x, w.double()), lambda: block_norm_forward(x, w, x.bfloat16()),
              lambda: dropout(x.double(), 0.5, 1), lambda: dropout(x, 0.5, 1, counter=torch.zeros(1, device="cuda"))):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: block_norm_forward(x, w, eps=0.0), lambda: dropout(x, 1.0, 1), lambda: dropout(x, -0.5, 1)):
        with pytest.raises(Shampoo4Error):
            f()


def test_captured_graph_draws_anew():
    """A captured training pass over two blocks, replayed with other work between: with the counter advanced the masks
    are those of the eager call at that count, and the same count gives the same bits."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward, dropout
    for t, c in ((700, 200), (40, 2200)):
        v = _case(t, c, "bf16", True, "channel", True, 0.0, 1.0)
        counter = torch.zeros(1, dtype=torch.int64, device="cuda")

        def call():
            kw = dict(post_weight=v["post"], gate=v["gate"], p=0.2, seed=3, offset=10, counter=counter)
            x0 = dropout(v["x"], 0.1, 3, 9, counter=counter)
            x, y, _, stats = block_norm_forward(x0, v["weight"], v["h"], **kw)
            return (x, y) + block_norm_backward(v["dy"], v["dres"], x, v["weight"], stats, h=v["h"], **kw)

        want = []
        for k in range(3):
            counter.fill_(k)
            want.append(call())
        assert not torch.equal(want[0][0], want[1][0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        announce(f"block graph {t}x{c}")
        with torch.cuda.stream(s):
            call()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = call()
        for k in (0, 2, 1, 1):
            for g in got:
                g.zero_()
            counter.fill_(k)
            torch.randn(1000, 1000, device="cuda").sum().item()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want[k], got))
