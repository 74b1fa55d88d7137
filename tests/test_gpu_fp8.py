"""e4m3 matrices with scales for blocks of 128 and the linear layer's product on them, on the GPU against
the float64 oracle.

Tolerances, u being the stored type's unit roundoff (bf16 2^-8, f16 2^-11, f32 2^-24):
* codes, scales and restored values are exact;
* a bf16 product: of eight neighbouring terms up to seven lose what is 13 bits below the largest's
  leading one, 7 2^-13 of the sum of sizes; then an fp32 addition (a rounding or a truncation) for each
  eight terms and for the at most 16 partial sums, (k / 8 + 18) 2^-23; and the store's rounding;
* an fp32 or f16 product: k exact terms and the partial sums added in fp32 in any order, (k + 18) 2^-23
  of the sum of sizes, and the store's rounding.
Terms and sums below 2^-126 may be lost: k 2^-126."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def _np(t):
    return t.detach().double().cpu().numpy()


def _rand(rng, t, c, dt, scale=1.0):
    x = scale * rng.standard_normal((t, c)) * np.exp(rng.standard_normal((1, c)))
    return torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dt])


def _strided(x, pad, offset=0):
    """The same values as a view with a larger leading dimension, starting `offset` elements in."""
    t, c = x.shape
    big = torch.full((t, c + pad + offset), float("nan"), dtype=x.dtype, device=x.device)
    big[:, offset:offset + c] = x
    return big[:, offset:offset + c]


def _same(a, codes, scales):
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    assert np.array_equal(a.codes.view(torch.uint8).cpu().numpy(), codes)


def _check_load(a, ref):
    from bit_quantized_shampoo_amd import fp8_load
    for dt in DT.values():
        y = fp8_load(a, dtype=dt)
        lim = 65504.0 if dt == torch.float16 else np.inf
        want = torch.from_numpy(np.clip(ref, -lim, lim).astype(np.float32)).to(dt)
        assert y.dtype == dt and torch.equal(torch.nan_to_num(y.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    out = torch.full((a.rows, a.cols + 7), 5.0, device="cuda")
    fp8_load(a, out=out[:, 3:3 + a.cols])
    assert torch.equal(torch.nan_to_num(out[:, 3:3 + a.cols]), torch.nan_to_num(fp8_load(a, torch.float32)))
    assert bool((out[:, :3] == 5).all()) and bool((out[:, 3 + a.cols:] == 5).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,c", [(1, 1), (1, 1024), (5, 7), (4, 128), (9, 129), (6, 513), (33, 300)])
def test_store_is_exact(t, c, dt):
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_store, fp8_store_weight
    x = _rand(np.random.default_rng(t * 1000 + c), t, c, dt)
    announce(f"fp8 store {t}x{c} {dt}")
    a = fp8_store(x)
    codes, scales = o.fp8_store(_np(x))
    _same(a, codes, scales)
    _check_load(a, o.fp8_load(codes, scales, c))
    _same(fp8_store(_strided(x, 5, 3)), codes, scales)
    codes, scales = o.fp8_store(_np(x), 128)
    tcodes, tscales = o.fp8_store(_np(x).T, 128)
    for v in (x, _strided(x, 4, 1)):
        w, wt = fp8_store_weight(v, transposed=True)
        _same(w, codes, scales)
        _same(wt, tcodes, tscales)
        _same(fp8_store_weight(v), codes, scales)
    _check_load(w, o.fp8_load(codes, scales, c, 128))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(127, 260), (128, 128), (129, 515), (300, 100)])
def test_store_weight_is_exact(n, k, dt):
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_store_weight
    rng = np.random.default_rng(n)
    w = _rand(rng, n, k, dt, 2.0 ** rng.integers(-40, 40))
    announce(f"fp8 weight {n}x{k} {dt}")
    a, b = fp8_store_weight(w, transposed=True)
    _same(a, *o.fp8_store(_np(w), 128))
    _same(b, *o.fp8_store(_np(w).T, 128))
    _check_load(b, o.fp8_load(*o.fp8_store(_np(w).T, 128), n, 128))


def test_store_special_values():
    """Zeros, subnormals, the power-of-two rule's edge, ties, the largest numbers, infinities and NaN in
    one block of several."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_store, fp8_store_weight
    rng = np.random.default_rng(5)
    x = np.zeros((24, 384), np.float32)
    x[1] = rng.standard_normal(384) * 1e-40
    x[2, :200] = 2.0 ** -126
    x[3, 0], x[3, 130] = 448.0, np.nextafter(np.float32(448), np.float32(449))
    x[4, :256] = np.concatenate([np.arange(128) + 0.5, np.arange(128) * 2.0 ** -10])
    x[5], x[6] = 3.4e38, -np.finfo(np.float32).max
    x[7] = rng.standard_normal(384)
    x[7, 200] = np.inf
    x[8] = rng.standard_normal(384)
    x[8, 5] = np.nan
    x[9] = -0.0
    x[10] = rng.standard_normal(384) * 2.0 ** rng.integers(-30, 8, 384)
    x[11, 0], x[12, 0], x[13, 383] = -np.inf, 1e-45, 65504.0
    for i in range(14, 24):
        x[i] = (rng.standard_normal(384) * 2.0 ** (12.0 * (i - 19))).astype(np.float32)
    announce("fp8 store special values")
    for dt in (torch.float32, torch.bfloat16):
        v = torch.from_numpy(x).cuda().to(dt)
        a = fp8_store(v)
        codes, scales = o.fp8_store(_np(v))
        _same(a, codes, scales)
        _check_load(a, o.fp8_load(codes, scales, 384))
    assert int(a.scales[7, 1]) == 255 and int(a.scales[7, 0]) != 255 and int(a.scales[8, 0]) == 255
    w, wt = fp8_store_weight(v, transposed=True)
    _same(w, *o.fp8_store(_np(v), 128))
    _same(wt, *o.fp8_store(_np(v).T, 128))


def test_store_offsets_beyond_32_bits():
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_load, fp8_store, fp8_store_weight
    ld = (1 << 31) // 32 + 64
    announce("fp8 store with 64-bit offsets")
    big = torch.zeros((40, ld), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(40, 50, device="cuda").bfloat16()
    big[:, -50:] = x
    for f in (fp8_store, fp8_store_weight):
        a, b = f(big[:, -50:]), f(x)
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)
    fp8_load(a, out=big[:, -50:])
    assert torch.equal(big[:, -50:], fp8_load(a)) and float(big[:, :-50].abs().amax()) == 0


def _check_linear(x, w, out_dt, quantised, base=None, pad=0, where=""):
    """fp8_linear against the oracle's product of the quantised operands (checked for themselves above)."""
    from bit_quantized_shampoo_amd import fp8_linear, fp8_load, fp8_store, fp8_store_weight
    (t, k), n = x.shape, w.shape[0]
    x8, w8 = fp8_store(x), fp8_store_weight(w)
    xv, wv = fp8_load(x8, torch.float32).double(), fp8_load(w8, torch.float32).double()
    ref, size = xv @ wv.t().contiguous(), xv.abs() @ wv.abs().t().contiguous()
    out = None
    if base is not None or pad:
        out = torch.full((t, n + pad + 2), 3.0, dtype=DT[out_dt], device="cuda")
        if base is not None:
            out[:, 1:1 + n] = base
            ref, size = ref + out[:, 1:1 + n].double(), size + out[:, 1:1 + n].double().abs()
    announce(f"fp8 linear {t}x{k} by {n}x{k} {x.dtype} -> {out_dt} quantised={quantised} added={base is not None} {where}")
    y = fp8_linear(x8 if quantised else x, w8, out=None if out is None else out[:, 1:1 + n],
                   accumulate=base is not None, dtype=DT[out_dt])
    torch.cuda.synchronize()
    if out is not None:
        assert bool((out[:, 0] == 3).all()) and bool((out[:, 1 + n:] == 3).all())
    assert y.dtype == DT[out_dt]
    e = 7 * 2.0 ** -13 + (k / 8 + 18) * 2.0 ** -23 if out_dt == "bf16" else (k + 18) * 2.0 ** -23
    tol = e * size * (1 + U[out_dt]) + U[out_dt] * ref.abs() + TINY[out_dt] + k * 2.0 ** -126
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), ((y.double() - ref).abs() / tol).amax())
    return y


@pytest.mark.parametrize("out_dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,n,k", [
    (1, 1, 1), (1, 16, 128), (1, 333, 1000), (1, 4096, 4096), (3, 130, 129), (8, 1024, 1024), (16, 17, 640), (17, 64, 96),
    (33, 200, 257), (64, 4096, 1024), (65, 129, 1153), (100, 1000, 300), (128, 128, 128), (129, 130, 2309), (257, 300, 513),
    (300, 256, 4096), (513, 1025, 384),
])
def test_linear(t, n, k, out_dt):
    require_gpu()
    rng = np.random.default_rng(t + n + k)
    x, w = _rand(rng, t, k, out_dt, 3.0), _rand(rng, n, k, "f32", 0.1)
    for quantised in (False, True):
        _check_linear(x, w, out_dt, quantised)
    base = _rand(rng, t, n, out_dt)
    _check_linear(_strided(x, 3, 1), w, out_dt, False, base=base, pad=5)


@pytest.mark.parametrize("dt,out_dt", [("f32", "bf16"), ("bf16", "f32"), ("f16", "bf16"), ("f32", "f16")])
def test_linear_mixed_types(dt, out_dt):
    require_gpu()
    rng = np.random.default_rng(8)
    for t in (5, 90):
        _check_linear(_rand(rng, t, 700, dt), _rand(rng, 210, 700, "f32", 0.1), out_dt, False)


@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
def test_linear_large_tiles(out_dt):
    """Sizes that take the largest tiles, whole and ragged, and sums split over long rows."""
    require_gpu()
    rng = np.random.default_rng(12)
    # 128 x 128 tiles (two), 256 x 256 (three, an odd number of blocks of k among them), ranges of k
    for t, n, k in ((2048, 2048, 256), (2049, 2500, 200), (4096, 4096, 1100), (4095, 4090, 1153), (3841, 4000, 4000),
                    (256, 256, 8192), (700, 300, 16400)):
        x = torch.randn(t, k, device="cuda").to(DT[out_dt])
        w = torch.randn(n, k, device="cuda") * 0.05
        _check_linear(x, w, out_dt, True, base=torch.randn(t, n, device="cuda").to(DT[out_dt]), pad=1)
        _check_linear(x, w, out_dt, True)


@pytest.mark.parametrize("t", [4, 80, 300, 2304])
@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
def test_linear_scales(t, out_dt):
    """Blocks whose scales lie far apart, at fp32's ends, zero rows; a block that is not finite makes the
    outputs that it enters NaN and no others."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store, fp8_store_weight
    g = torch.Generator(device="cuda").manual_seed(t)
    n, k = (2304 if t == 2304 else 300), 600
    x = torch.randn(t, k, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (t, 5), generator=g, device="cuda").float()).repeat_interleave(128, 1)[:, :k]
    x[1] = 0
    w = torch.randn(n, k, generator=g, device="cuda")
    w *= torch.exp2(torch.randint(-20, 20, (1, 5), generator=g, device="cuda").float()).repeat_interleave(128, 1)[:, :k]
    _check_linear(x, w, out_dt, True, where="scales")
    _check_linear(x * 2.0 ** 90, w * 2.0 ** -90, out_dt, True, where="large by small")
    _check_linear(x * 2.0 ** -95, w * 2.0 ** 90, out_dt, True, where="small by large")
    _check_linear(x * 2.0 ** -80, w * 2.0 ** -30, out_dt, True, where="towards the smallest numbers")
    x[2, 130], w[140, 300] = float("nan"), float("inf")
    announce(f"fp8 linear with NaN {t}")
    y = fp8_linear(fp8_store(x), fp8_store_weight(w), dtype=DT[out_dt])
    bad = torch.zeros(t, n, dtype=torch.bool, device="cuda")
    bad[2] = True
    bad[:, 128:256] = True
    assert torch.equal(torch.isnan(y), bad)


def test_linear_not_finite_on_the_largest_tiles():
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store, fp8_store_weight
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = torch.randn(4000, 1160, generator=g, device="cuda"), torch.randn(4090, 1160, generator=g, device="cuda")
    want = fp8_linear(fp8_store(x), fp8_store_weight(w), dtype=torch.bfloat16)
    x[3999, 1159], w[256, 0] = float("inf"), float("nan")
    announce("fp8 linear with NaN on the largest tiles")
    y = fp8_linear(fp8_store(x), fp8_store_weight(w), dtype=torch.bfloat16)
    bad = torch.zeros(4000, 4090, dtype=torch.bool, device="cuda")
    bad[3999] = True
    bad[:, 256:384] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("t,n,k", [(16384, 4096, 256), (16130, 4090, 300), (12289, 5000, 1160), (16384, 4096, 700)])
def test_linear_many_large_tiles(t, n, k):
    """More tiles than CUs, one after the other in a workgroup: what rows give does not depend on how many are with
    them, to the last bit, and the oracle holds on some of them.  Edges, odd numbers of blocks, added, odd strides."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_load, fp8_store, fp8_store_weight
    g = torch.Generator(device="cuda").manual_seed(t + k)
    x = torch.randn(t, k, generator=g, device="cuda").bfloat16()
    w8 = fp8_store_weight(torch.randn(n, k, generator=g, device="cuda"))
    announce(f"fp8 linear of many large tiles {t}x{n}x{k}")
    y = fp8_linear(x, w8)
    for i in range(0, t, 1000):
        assert torch.equal(y[i:i + 1000], fp8_linear(x[i:i + 1000].contiguous(), w8)), i
    wd = fp8_load(w8, dtype=torch.float32).double().cpu()
    for i in (0, 255, 256, 8191, t - 1):
        xd = fp8_load(fp8_store(x[i:i + 1]), dtype=torch.float32).double().cpu()
        ref, size = (xd @ wd.T)[0], (xd.abs() @ wd.abs().T)[0]
        assert bool(((y[i].double().cpu() - ref).abs() <= 7 * 2.0 ** -13 * size + 2.0 ** -8 * ref.abs() + 1e-30).all()), i
    for ld in (n + 8, n + 1):
        out = torch.full((t, ld), 0.5, dtype=torch.bfloat16, device="cuda")
        for _ in range(2):
            fp8_linear(x, w8, out=out[:, :n], accumulate=True)
        want = torch.full((t, n), 0.5, dtype=torch.bfloat16, device="cuda")
        for i in range(0, t, 1000):
            for _ in range(2):
                fp8_linear(x[i:i + 1000].contiguous(), w8, out=want[i:i + 1000], accumulate=True)
        assert torch.equal(out[:, :n], want) and bool((out[:, n:] == 0.5).all())


def test_linear_into_its_input_is_refused():
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store_weight
    x = torch.randn(5, 64, device="cuda").bfloat16()
    w8 = fp8_store_weight(torch.randn(64, 64, device="cuda"))
    announce("fp8 linear into its input")
    with pytest.raises(ValueError):
        fp8_linear(x, w8, out=x)
    with pytest.raises(ValueError):
        fp8_linear(x, w8, out=x, accumulate=True)


def test_linear_does_not_depend_on_other_rows():
    """Rows behind the last and columns behind the last weight row are neither read nor written."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store_weight
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (3, 70, 260):
        x = torch.randn(t + 9, 300, generator=g, device="cuda").bfloat16()
        w8 = fp8_store_weight(torch.randn(77, 300, generator=g, device="cuda"))
        want = fp8_linear(x[:t].clone(), w8)
        x[t:] = float("nan")
        out = torch.full((t + 9, 80), 2.0, dtype=torch.bfloat16, device="cuda")
        announce(f"fp8 linear rows {t}")
        fp8_linear(x[:t], w8, out=out[:t, :77])
        assert torch.equal(out[:t, :77], want)
        assert bool((out[t:] == 2).all()) and bool((out[:, 77:] == 2).all())


def test_no_rows():
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_load, fp8_store, fp8_store_weight
    announce("fp8 without rows")
    x = torch.empty(0, 70, device="cuda")
    a = fp8_store(x)
    assert fp8_load(a).shape == (0, 70)
    w8, wt8 = fp8_store_weight(torch.randn(5, 70, device="cuda"), transposed=True)
    assert fp8_linear(x, w8).shape == (0, 5) and fp8_linear(a, w8).shape == (0, 5)
    with pytest.raises(ValueError):
        fp8_linear(x, wt8)


def test_binding_refusals():
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store, fp8_store_weight
    x, w = torch.zeros(4, 130, device="cuda"), torch.zeros(6, 130, device="cuda")
    x8, w8 = fp8_store(x), fp8_store_weight(w)
    for f in (lambda: fp8_linear(x, x8), lambda: fp8_linear(w8, w8), lambda: fp8_linear(x[:, :128], w8),
              lambda: fp8_linear(x, w8, accumulate=True), lambda: fp8_linear(x, w8, out=torch.zeros(4, 5, device="cuda")),
              lambda: fp8_linear(x.t(), w8), lambda: fp8_store(x.t()), lambda: fp8_store(x, out=w8),
              lambda: fp8_store_weight(w, out_t=w8), lambda: fp8_store_weight(w, transposed=True, out_t=w8)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fp8_linear(x, w), lambda: fp8_linear(x, w8, dtype=torch.float64), lambda: fp8_linear(x.double(), w8),
              lambda: fp8_linear(x, w8, out=torch.zeros(4, 6, device="cuda"), dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            f()


def test_gradient_is_the_difference():
    """<dy, (layer(x + h d) - layer(x))> = <fp8_linear(dy, wt8), h d> for operands that the format holds
    exactly (small integers): both sides are exact sums of integers."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store_weight
    g = torch.Generator(device="cuda").manual_seed(3)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()  # noqa: E731
    for t in (7, 150):
        x, d, w, dy = ints(t, 200), ints(t, 200), ints(170, 200), ints(t, 170)
        w8, wt8 = fp8_store_weight(w, transposed=True)
        announce(f"fp8 linear differences {t}")
        for dt in (torch.float32, torch.bfloat16):
            change = fp8_linear((x + d).to(dt), w8, dtype=torch.float32) - fp8_linear(x.to(dt), w8, dtype=torch.float32)
            dx = fp8_linear(dy.to(dt), wt8, dtype=torch.float32)
            assert float((dy.double() * change.double()).sum()) == float((dx.double() * d.double()).sum())


def test_captured_graphs_and_streams():
    """A layer's forward and backward products from a captured graph, replayed with other work between the
    replays, and on a stream given, against the eager results."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store_weight
    g = torch.Generator(device="cuda").manual_seed(9)
    for t, n, k in ((4, 300, 500), (300, 260, 1000), (2304, 2304, 300)):
        x, dy = (torch.randn(t, c, generator=g, device="cuda").bfloat16() for c in (k, n))
        w = torch.randn(n, k, generator=g, device="cuda")

        def call():
            w8, wt8 = fp8_store_weight(w, transposed=True)
            return fp8_linear(x, w8), fp8_linear(dy, wt8)

        want = call()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        announce(f"fp8 graph {t} {n} {k}")
        with torch.cuda.stream(s):
            call()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = call()
        for _ in range(3):
            for v in got:
                v.zero_()
            torch.randn(1000, 1000, device="cuda").sum().item()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        again = fp8_linear(x, fp8_store_weight(w, stream=s), stream=s)
        s.synchronize()
        assert torch.equal(again, want[0])
