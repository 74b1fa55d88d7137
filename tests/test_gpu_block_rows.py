"""The ends of a residual block on the GPU: rows that are not finite, more rows than a workgroup has at once in every
form of the backward kernel, in-place calls without a norm behind the block, and offsets beyond 32 bits.

Tolerances are those of test_gpu_block.py, whose check against the oracle is used here; what is compared with another
call of the same kernels is compared bit for bit."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_block import DT, E, OFFSET, OPTIONS, SEED, TINY, U, _case, _check, _close, _np, _rand, _vec

pytestmark = pytest.mark.gpu


def _same_codes(a, b):
    assert torch.equal(a.scales, b.scales), np.argwhere((a.scales != b.scales).cpu().numpy())[:4].tolist()
    assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("c", [3, 130, 600, 1030, 2309, 4100, 8200])
def test_codes_of_rows_that_are_not_finite(c, dt):
    """A NaN or an infinity in x or h: y8 is what storing y gives, its padding (code 0, scale byte 1) with it."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_forward, fp8_store
    rng = np.random.default_rng(c)
    w, post = _vec(rng, c, 1.0), _vec(rng, c, 0.5)
    x, h = _rand(rng, 9, c, dt), _rand(rng, 9, c, dt)
    x[1, c // 2], x[2, 0], h[4, c - 1], h[5, 1] = float("nan"), float("inf"), float("nan"), float("-inf")
    x[7] = float("nan")
    announce(f"codes of rows that are not finite {c} {dt}")
    for kw in (dict(), dict(h=h), dict(h=h, post_weight=post), dict(h=h, post_weight=post, p=0.3, seed=1)):
        _, y, y8, _ = block_norm_forward(x, w, save8=True, **kw)
        assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[7]).all())
        assert bool(torch.isfinite(y[[0, 3, 6, 8]]).all())
        _same_codes(y8, fp8_store(y))
        assert bool((y8.scales[:, -(-c // 128):] == 1).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,c,p", [(64, 3, 0.8), (64, 9, 0.9), (16, 129, 1 - 2.0 ** -16), (8, 1030, 1 - 2.0 ** -16)])
def test_dropped_rows_that_are_not_finite(t, c, p, dt):
    """A block's end that is NaN as a whole (a NaN before the norm behind the block), of which dropout keeps nothing in
    some rows: there x' is the residual alone, and its norm is that of any other row."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_forward, fp8_store
    rng = np.random.default_rng(t + c)
    x, h, w, post = _rand(rng, t, c, dt), _rand(rng, t, c, dt), _vec(rng, c, 1.0), _vec(rng, c, 0.5)
    h[:, c // 2] = float("nan")
    gone = ~o.dropout_keep(t, c, np.float32(p), SEED, OFFSET).any(1)
    assert gone.sum() >= t // 4
    announce(f"dropped rows that are not finite {t}x{c} {dt} p={p}")
    for gate in (None, _vec(rng, c, 0.6), _rand(rng, t, c, dt, 0.5)):
        xn, y, y8, stats = block_norm_forward(x, w, h, post_weight=post, gate=gate, p=p, seed=SEED, offset=OFFSET,
                                              eps=1e-5, save8=True)
        alone, ya, _, sa = block_norm_forward(x, w, eps=1e-5)
        rows = torch.from_numpy(gone).cuda()
        assert torch.equal(xn[rows], x[rows]) and torch.equal(y[rows], ya[rows])
        assert torch.equal(stats[1][rows], sa[1][rows]) and bool(torch.isnan(stats[1][~rows]).all())
        r = o.rstd(_np(x), float(np.float32(1e-5)))[gone]
        ref = _np(x)[gone] * r * _np(w)
        _close(y[rows], ref, (36 * E + U[dt]) * np.abs(ref) + TINY[dt], "y")
        _same_codes(y8, fp8_store(y))


@pytest.mark.parametrize("t,c,dt,options", [
    (2100, 400, "f32", OPTIONS[1]), (2100, 1000, "bf16", OPTIONS[4]), (1030, 2048, "f16", OPTIONS[2]),
    (1100, 4096, "bf16", (True, "channel", True, 0.0, 1.0)), (600, 3001, "f32", (True, "token", True, 0.0, 0.5)),
    (530, 8192, "bf16", (False, "channel", True, 0.0, 1.0)), (259, 5000, "f32", (True, "channel", True, 0.0, 0.9)),
    (520, 4096, "bf16", (True, "channel", True, 0.1, 1.0)),
])
def test_more_rows_than_workgroups(t, c, dt, options):
    """A wave, or a workgroup, has a second row in every form of the backward kernel, some of them one more than others:
    rows a workgroup has at once are 2048 up to 1024 columns, 1024 up to 2048, 512 up to 4096 and 256 up to 8192."""
    require_gpu()
    _check(t, c, dt, *options)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("c", [5, 515, 2309, 4099, 8203])
def test_in_place_without_a_norm_behind(c, gate, dt):
    """Nothing makes a row's waves meet before its first result is written."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward
    for weight, p in ((True, 0.0), (False, 0.2)):
        v = _case(5, c, dt, False, gate, weight, 0.0, 0.5)
        kw = dict(gate=v["gate"], residual_scale=0.5, p=p, seed=SEED, offset=OFFSET)
        announce(f"block in place {c} {dt} gate={gate} weight={weight}")
        x, y, _, stats = block_norm_forward(v["x"], v["weight"], v["h"], **kw)
        got = block_norm_backward(v["dy"], v["dres"], x, v["weight"], stats, h=v["h"], **kw)
        for target in ("x", "h"):
            a = {k: v[k].clone() for k in ("x", "h")}
            x2, y2, _, _ = block_norm_forward(a["x"], v["weight"], a["h"], out=a[target], **kw)
            assert x2 is a[target] and torch.equal(x2, x) and (y is None or torch.equal(y2, y))
        if weight:
            h = v["h"].clone()
            x2, _, _, _ = block_norm_forward(v["x"], v["weight"], h, y=h, **kw)
            assert torch.equal(x2, x) and torch.equal(h, y)
        for tx, th in (("dres", "h"), ("dy", "dres"), ("dres", "dy")):
            if not weight and "dy" in (tx, th):
                continue
            a = {k: None if v[k] is None else v[k].clone() for k in ("dy", "dres", "h")}
            again = block_norm_backward(a["dy"], a["dres"], x, v["weight"], stats, h=a["h"], dx=a[tx], dh=a[th], **kw)
            assert all((q is None and r is None) or torch.equal(q, r) for q, r in zip(got, again))


@pytest.mark.parametrize("t,c", [(40, 50), (5, 1030), (9, 9000)])
def test_offsets_beyond_32_bits(t, c):
    """Every matrix of both calls as columns of one long one, its last rows more than 2^31 elements from the first."""
    require_gpu()
    from bit_quantized_shampoo_amd import block_norm_backward, block_norm_forward
    v = _case(t, c, "bf16", True, "token", True, 0.0, 1.0)
    kw = dict(post_weight=v["post"], residual_scale=0.5, p=0.1, seed=SEED, offset=OFFSET)
    x, y, _, stats = block_norm_forward(v["x"], v["weight"], v["h"], gate=v["gate"], **kw)
    want = block_norm_backward(v["dy"], v["dres"], x, v["weight"], stats, h=v["h"], gate=v["gate"], **kw)
    names = ("x", "h", "gate", "dy", "dres", "out", "y", "dx", "dh")
    big = torch.empty((t, (1 << 31) // (t - 1) * 9 // 8 + len(names) * c), dtype=DT["bf16"], device="cuda")
    m = {k: big[:, big.shape[1] - (i + 1) * c:big.shape[1] - i * c] for i, k in enumerate(names)}
    for k in names[:5]:
        m[k].copy_(v[k])
    announce(f"block {t}x{c}, rows {big.shape[1]} apart")
    x2, y2, _, s2 = block_norm_forward(m["x"], v["weight"], m["h"], gate=m["gate"], out=m["out"], y=m["y"], **kw)
    assert torch.equal(x2, x) and torch.equal(y2, y) and torch.equal(s2, stats)
    got = block_norm_backward(m["dy"], m["dres"], m["out"], v["weight"], s2, h=m["h"], gate=m["gate"], dx=m["dx"],
                              dh=m["dh"], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
