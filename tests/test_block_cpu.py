"""Host-only checks of the residual block's operators: every call refuses what the header says it refuses
before anything reaches a device, the binding checks its arguments, and the oracle is held against what
is known by other ways (the number formats' own properties, the generator's published test vectors,
differences of the forward formulas)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from bit_quantized_shampoo_amd import _lib as L
from bit_quantized_shampoo_amd import train as T
from oracle import train as o

P = 0x10000          # an aligned address that no refused call may touch


def _lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return L.lib()


# -- refusals ------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols,block,status,codes,scales", [
    (1, 1, 1, L.OK, 128, 4), (3, 513, 1, L.OK, 3 * 640, 3 * 8), (129, 128, 128, L.OK, 129 * 128, 2 * 4),
    (0, 5, 1, L.OK, 0, 0), (4, 4, 32, L.EINVAL, 0, 0), (-1, 4, 1, L.ESHAPE, 0, 0), (4, 0, 1, L.ESHAPE, 0, 0),
    (1 << 31, 4, 1, L.ESHAPE, 0, 0),
])
def test_fp8_bytes(rows, cols, block, status, codes, scales):
    c, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert _lib().shampoo4_fp8_bytes(rows, cols, block, ctypes.byref(c), ctypes.byref(s)) == status
    if status == L.OK:
        assert (c.value, s.value) == (codes, scales)
        shapes = T.Fp8.padded(rows, cols, block)
        assert (int(np.prod(shapes[0])), int(np.prod(shapes[1]))) == (codes, scales)


def test_fp8_store_and_load_refusals():
    lib = _lib()
    store, weight, load = lib.shampoo4_fp8_store, lib.shampoo4_fp8_store_weight, lib.shampoo4_fp8_load
    assert store(3, 4, 4, P, 4, P, P, None) == L.EINVAL
    assert store(L.F32, -1, 4, P, 4, P, P, None) == L.ESHAPE
    assert store(L.F32, 4, 0, P, 4, P, P, None) == L.ESHAPE
    assert store(L.F32, 4, 4, P, 3, P, P, None) == L.ESHAPE
    assert store(L.F32, 4, 4, None, 4, P, P, None) == L.EINVAL
    assert store(L.F32, 4, 4, P, 4, None, P, None) == L.EINVAL
    assert store(L.F32, 4, 4, P, 4, P, None, None) == L.EINVAL
    assert store(L.F32, 4, 4, P + 2, 4, P, P, None) == L.EALIGN
    assert store(L.BF16, 4, 4, P, 4, P + 8, P, None) == L.EALIGN
    assert store(L.BF16, 4, 4, P, 4, P, P + 2, None) == L.EALIGN
    assert store(L.BF16, 1 << 30, 1 << 30, P, 1 << 30, P, P, None) == L.ESHAPE
    assert store(L.F32, 0, 4, None, 4, None, None, None) == L.OK
    assert weight(L.F32, 4, 4, P, 4, P, P, P, None, None) == L.EINVAL          # half of the transposed pair
    assert weight(L.F32, 4, 4, P, 4, P, P, None, P, None) == L.EINVAL
    assert weight(L.F32, 4, 4, P, 4, P, P, P + 4, P, None) == L.EALIGN
    assert weight(L.F32, 4, 4, P, 4, None, None, P, P, None) == L.EINVAL
    assert weight(L.F32, 1 << 20, 1 << 20, P, 1 << 20, P, P, None, None, None) == L.ESHAPE
    assert weight(L.F32, 0, 4, None, 4, None, None, None, None, None) == L.OK
    assert load(L.F16, 4, 4, 2, P, P, P, 4, None) == L.EINVAL
    assert load(L.F16, 4, 4, 1, None, None, P, 4, None) == L.EINVAL
    assert load(L.F16, 4, 4, 128, P, P, P, 2, None) == L.ESHAPE
    assert load(L.F16, 0, 4, 1, None, None, None, 4, None) == L.OK


def test_linear_refusals():
    lib = _lib()
    f = lib.shampoo4_fp8_linear
    big = 1 << 20

    def call(dtype=L.BF16, odtype=L.BF16, rows=4, n=8, k=16, x=None, ldx=0, xc=P, xs=P, wc=P, ws=P, acc=0, y=P, ldy=8,
             wk=None, wb=0):
        return f(dtype, odtype, rows, n, k, x, ldx, xc, xs, wc, ws, acc, y, ldy, wk, wb, None)

    assert call(dtype=7) == L.EINVAL and call(odtype=-1) == L.EINVAL
    assert call(x=P, ldx=16) == L.EINVAL                          # x twice
    assert call(xc=None, xs=None) == L.EINVAL and call(xs=None) == L.EINVAL
    assert call(x=P, ldx=15, xc=None, xs=None) == L.ESHAPE
    assert call(x=P + 1, ldx=16, xc=None, xs=None) == L.EALIGN
    assert call(wc=None) == L.EINVAL and call(ws=None) == L.EINVAL and call(y=None) == L.EINVAL
    assert call(wc=P + 8) == L.EALIGN and call(xc=P + 8) == L.EALIGN and call(ws=P + 1) == L.EALIGN
    assert call(y=P + 1) == L.EALIGN and call(ldy=7) == L.ESHAPE
    assert call(n=0) == L.ESHAPE and call(k=0) == L.ESHAPE and call(rows=-1) == L.ESHAPE
    assert call(rows=big * 8, n=big * 8, ldy=big * 8) == L.ESHAPE
    assert call(rows=0, xc=None, xs=None, wc=None, ws=None, y=None) == L.OK
    need = lib.shampoo4_fp8_linear_workspace_bytes(L.BF16, 200, 8, 16, 0)
    assert need >= 200 * (128 + 4)
    given = dict(rows=200, x=P, ldx=16, xc=None, xs=None)
    assert call(**given) == L.EINVAL and call(**given, wk=P, wb=need - 1) == L.ESMALLBUF
    assert call(**given, wk=P + 16, wb=need) == L.EALIGN
    assert lib.shampoo4_fp8_linear_workspace_bytes(L.BF16, 200, 0, 16, 0) == 0
    assert lib.shampoo4_fp8_linear_workspace_bytes(9, 200, 8, 16, 0) == 0


def test_dropout_refusals():
    f = _lib().shampoo4_dropout

    def call(p=0.5, reserved=0, counter=None, dtype=L.F32, rows=4, cols=4, x=P, ldx=4, y=P, ldy=4):
        cfg = L.DropoutConfig(p, reserved, 1, 2, counter)
        return f(ctypes.byref(cfg), dtype, rows, cols, x, ldx, y, ldy, None)

    for bad in (-0.1, 1.0, 1.0 - 2.0 ** -18, 1.5, float("nan"), float("inf")):
        assert call(p=bad) == L.EINVAL, bad
    assert call(reserved=1) == L.EINVAL and call(dtype=4) == L.EINVAL
    assert call(counter=P + 4) == L.EALIGN
    assert call(x=None) == L.EINVAL and call(y=None) == L.EINVAL
    assert call(ldx=3) == L.ESHAPE and call(ldy=3) == L.ESHAPE and call(cols=0) == L.ESHAPE and call(rows=-1) == L.ESHAPE
    assert call(rows=1 << 30, cols=1 << 20, ldx=1 << 20, ldy=1 << 20) == L.ESHAPE
    assert f(None, L.F32, 4, 4, P, 4, P, 4, None) == L.EINVAL
    assert call(rows=0, x=None, y=None) == L.OK


def _config(eps=1e-6, rho=1.0, p=0.0):
    return L.BlockNormConfig(eps, rho, L.DropoutConfig(p, 0, 0, 0, None))


def test_block_forward_refusals():
    f = _lib().shampoo4_block_norm_forward

    def call(cfg=None, dtype=L.F32, rows=4, cols=8, x=P, ldx=8, h=P, ldh=8, post=P, gate=P, grows=0, ldg=0, weight=P,
             out=P, ldo=8, y=P, ldy=8, yc=None, ys=None, hr=P, r=P):
        c = cfg or _config()
        return f(ctypes.byref(c), dtype, rows, cols, x, ldx, h, ldh, post, gate, grows, ldg, weight, out, ldo, y, ldy, yc,
                 ys, hr, r, None)

    for bad in (_config(eps=0.0), _config(eps=1e-31), _config(eps=float("inf")), _config(eps=float("nan")),
                _config(rho=float("nan")), _config(p=1.0)):
        assert call(cfg=bad) == L.EINVAL
    assert f(None, L.F32, 4, 8, P, 8, P, 8, P, P, 0, 0, P, P, 8, P, 8, None, None, P, P, None) == L.EINVAL
    assert call(dtype=8) == L.EINVAL and call(grows=2) == L.EINVAL
    assert call(cols=0) == L.ESHAPE and call(cols=16385) == L.ESHAPE and call(rows=1 << 24) == L.ESHAPE
    assert call(rows=-1) == L.ESHAPE
    for cols, most in ((2048, 1 << 24), (2049, 1 << 23), (4096, 1 << 23), (4097, 1 << 22)):      # of one launch
        wide = dict(cols=cols, ldx=cols, ldh=cols, ldo=cols, ldy=cols)
        assert call(**wide, rows=most) == L.ESHAPE and call(**wide, rows=most - 1, x=None) == L.EINVAL
    for k in ("ldx", "ldh", "ldo", "ldy"):
        assert call(**{k: 7}) == L.ESHAPE, k
    assert call(grows=1, ldg=7) == L.ESHAPE and call(grows=1, ldg=8, gate=None) == L.EINVAL
    for k in ("x", "out"):
        assert call(**{k: None}) == L.EINVAL, k
    assert call(y=None) == L.EINVAL                               # weight without a result
    assert call(weight=None) == L.EINVAL                          # results without weight
    assert call(yc=P) == L.EINVAL and call(ys=P) == L.EINVAL
    assert call(yc=P + 8, ys=P) == L.EALIGN
    for k in ("post", "gate", "weight", "hr", "r"):
        assert call(**{k: P + 2}) == L.EALIGN, k
    alone = dict(h=None, post=None, gate=None, out=None, hr=None)
    for k, v in (("post", P), ("gate", P), ("out", P), ("hr", P), ("grows", 1), ("cfg", _config(rho=0.5))):
        assert call(**{**alone, k: v}) == L.EINVAL, k
    assert call(**alone, weight=None, y=None, r=None) == L.EINVAL # nothing to do
    assert call(rows=0, x=None, h=None, out=None, y=None) == L.OK


def test_block_backward_refusals():
    lib = _lib()
    f = lib.shampoo4_block_norm_backward
    need = lib.shampoo4_block_norm_workspace_bytes(4, 8)
    assert need >= 3 * 8 * 4

    def call(cfg=None, dtype=L.F32, rows=4, cols=8, dy=P, lddy=8, dres=P, lddres=8, x=P, ldx=8, r=P, weight=P, h=P, ldh=8,
             hr=P, post=P, gate=P, grows=0, ldg=0, dx=P, lddx=8, dh=P, lddh=8, dw=P, dp=P, dg=P, lddg=0, ws=P, wsb=need):
        c = cfg or _config()
        return f(ctypes.byref(c), dtype, rows, cols, dy, lddy, dres, lddres, x, ldx, r, weight, h, ldh, hr, post, gate,
                 grows, ldg, dx, lddx, dh, lddh, dw, dp, dg, lddg, ws, wsb, None)

    assert call(cfg=_config(eps=-1.0)) == L.EINVAL and call(cfg=_config(p=2.0)) == L.EINVAL and call(dtype=3) == L.EINVAL
    assert call(cols=16385) == L.ESHAPE and call(rows=-1) == L.ESHAPE
    for k in ("lddy", "lddres", "ldx", "ldh", "lddx", "lddh"):
        assert call(**{k: 7}) == L.ESHAPE, k
    for k in ("dy", "r", "x", "hr"):
        assert call(**{k: None}) == L.EINVAL, k
    assert call(weight=None) == L.EINVAL                          # dy without weight
    none = dict(weight=None, dy=None, r=None, dw=None)
    assert call(**none, dres=None) == L.EINVAL
    assert call(post=None) == L.EINVAL and call(gate=None) == L.EINVAL
    alone = dict(h=None, hr=None, post=None, gate=None, dh=None, dp=None, dg=None)
    for k, v in (("post", P), ("gate", P), ("hr", P), ("dh", P), ("dp", P), ("dg", P), ("cfg", _config(rho=2.0))):
        assert call(**{**alone, k: v}) == L.EINVAL, k
    assert call(grows=1, ldg=7) == L.ESHAPE and call(grows=1, ldg=8, lddg=7) == L.ESHAPE and call(grows=3) == L.EINVAL
    assert call(wsb=need - 1) == L.ESMALLBUF and call(ws=None) == L.EINVAL and call(ws=P + 8) == L.EALIGN
    for k in ("r", "weight", "hr", "post", "gate", "dw", "dp", "dg"):
        assert call(**{k: P + 2}) == L.EALIGN, k
    assert lib.shampoo4_block_norm_workspace_bytes(4, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x, v = torch.zeros(4, 8), torch.zeros(8)
    for f in (lambda: T.fp8_store(x), lambda: T.fp8_store_weight(x), lambda: T.fp8_load(None), lambda: T.fp8_linear(x, None),
              lambda: T.dropout(x, 0.1, 0), lambda: T.block_norm_forward(x, v),
              lambda: T.block_norm_backward(x, x, x, v, torch.zeros(2, 4)), lambda: T.Fp8.empty(4, 8, device="cpu")):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError):
        T.Fp8(x, x, 4, 8, 64)
    assert T.Fp8.padded(3, 129) == ((3, 256), (3, 4)) and T.Fp8.padded(129, 513, 128) == ((129, 640), (2, 8))


# -- the oracle ----------------------------------------------------------------------------

def test_oracle_e4m3_is_the_format():
    """Its numbers are those of torch's float8_e4m3fn, and the nearest one is found for values between."""
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = o.e4m3_value(codes)
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    assert np.array_equal(np.isnan(got), np.isnan(want))
    v = np.random.default_rng(0).uniform(-448, 448, 5000) * 2.0 ** np.random.default_rng(1).integers(-18, 1, 5000)
    back = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.e4m3_value(o.e4m3_code(v.astype(np.float32).astype(np.float64))), back)
    mid = (o.e4m3_numbers()[1:] + o.e4m3_numbers()[:-1]) / 2      # ties go to the even code
    assert np.all(o.e4m3_code(mid) % 2 == 0)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_oracle_fp8_properties(block_rows):
    """A value is within 2^-4 of itself or 2^-10 of its scale; values of the format are fixed points; the largest
    code of a block is above 224; a transposed weight has the same values."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((140, 300)) * 10.0 ** rng.uniform(-20, 20, (140, 1))
    codes, scales = o.fp8_store(x, block_rows)
    y = o.fp8_load(codes, scales, 300, block_rows)
    s = np.repeat(np.repeat(2.0 ** (scales.astype(float) - 127), block_rows, 0)[:140, :3], 128, 1)[:, :300]
    assert np.all(np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10))
    top = np.abs(y / s)
    for b in range(len(scales)):
        for j in range(3):
            assert 208 <= top[b * block_rows:(b + 1) * block_rows, 128 * j:128 * j + 128].max() <= 448
    c2, s2 = o.fp8_store(y, block_rows)
    assert np.array_equal(o.fp8_load(c2, s2, 300, block_rows), y)
    assert np.all(codes[:, 300:] == 0) and np.all(scales[:, 3:] == 1)
    if block_rows == 128:
        assert np.array_equal(o.fp8_load(*o.fp8_store(x.T, 128), 140, 128), y.T)


@pytest.mark.parametrize("counter,key,want", [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_oracle_generator_known_answers(counter, key, want):
    """The test vectors that its authors published."""
    assert o.philox(counter, key) == want


def test_oracle_dropout_keeps_the_right_share():
    """Of 8000 elements (1 - p) 8000 are kept, five standard deviations aside."""
    for p in (0.0, 0.1, 0.5):
        kept = o.dropout_keep(50, 160, p, 11, 5).sum()
        assert abs(kept - 8000 * (1 - p)) <= 5 * np.sqrt(8000 * p * (1 - p))
    a = o.dropout_keep(4, 24, 0.5, 11, 5)
    assert np.array_equal(a[2:, 8:], o.dropout_keep(2, 16, 0.5, 11, 5, row0=2, col0=8))
    assert not np.array_equal(a, o.dropout_keep(4, 24, 0.5, 11, 6))
    assert not np.array_equal(a, o.dropout_keep(4, 24, 0.5, 12, 5))


@pytest.mark.parametrize("post,gate,weight", [(True, "channel", True), (False, "token", True), (True, None, False),
                                              (False, "channel", True), (True, "token", False)])
def test_oracle_block_gradients_are_differences(post, gate, weight):
    """Every gradient against central differences of sum(dy y) + sum(dres x'), of float64 formulas whose own
    error is about 1e-9."""
    rng = np.random.default_rng(4)
    t, c, rho, eps = 3, 10, 0.7, 1e-3
    v = {"x": rng.standard_normal((t, c)), "h": rng.standard_normal((t, c))}
    if post:
        v["post"] = rng.standard_normal(c)
    if gate:
        v["gate"] = rng.standard_normal(c if gate == "channel" else (t, c))
    if weight:
        v["weight"] = rng.standard_normal(c)
    drop = o.dropout_keep(t, c, 0.3, 1, 2) * o.dropout_scale(0.3)
    dy, dres = rng.standard_normal((t, c)) if weight else None, rng.standard_normal((t, c))

    def loss(v):
        x = o.block_end(v["x"], v["h"], v.get("post"), v.get("gate"), drop, rho, eps)
        return np.sum(dres * x) + (np.sum(dy * x * o.rstd(x, eps) * v["weight"]) if weight else 0.0)

    x = o.block_end(v["x"], v["h"], v.get("post"), v.get("gate"), drop, rho, eps)
    got, size = o.block_backward(dy, dres, x, v.get("weight"), v["h"], v.get("post"), v.get("gate"), drop, rho, eps)
    got = {"x": got["dx"], "h": got["dh"], "post": got["dpost"], "weight": got.get("dweight"),
           "gate": got["dgate"].sum(0) if gate == "channel" else got["dgate"]}
    for name, value in v.items():
        for i in np.ndindex(value.shape):
            up, down = {**v, name: value.copy()}, {**v, name: value.copy()}
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - got[name][i]) < 1e-7, (name, i)
    assert all(np.all(size[k] >= 0) for k in size)
