"""The ends of a residual block on the GPU: rows that are not finite.

Tolerances are those of test_gpu_block.py; what is compared with another call of the framework is compared bit for
bit."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_block import E, OFFSET, SEED, TINY, U, _close, _np, _rand, _vec

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
