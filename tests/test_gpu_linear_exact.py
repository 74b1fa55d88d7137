"""The linear layer's product on operands whose products and sums are exact, on the GPU: every output has to be the
rounded integer, bit for bit, so that a term lost, taken twice or scaled wrongly shows.

x and w are integers of size at most 3 times powers of two: one for each block of 128 columns (2^0 to 2^3 in x, 2^0 to
2^2 in w), one for each row of x (2^0 to 2^4) and one for each 128 rows of w (2^0 or 2^1).  Integers up to 16 are
numbers of e4m3 whatever power of two their block's scale is, so storing rounds nothing.  The products of a block lie
between 1 and 9 of one unit, less than four bits apart, where the 8-bit cores cut 13 bits below the largest.  But for
the factors of its row and its column every partial sum is an integer of at most 9 * 2^5 * k < 2^24 for k < 58254,
exact in float32 in any order (longer sums: x of 0 and +-1, few of them not 0).  What is left is the store's one
rounding, to nearest even, which `to(dtype)` does too."""

import pytest
import torch

from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _powers(n, m, step):
    """2^(step (i / 128) mod m), for i < n."""
    return torch.exp2(((torch.arange(n, device="cuda") // 128 * step) % m).float())


def _operands(t, n, k, dt):
    """x of type dt and w float32, and their product as float32."""
    g = torch.Generator(device="cuda").manual_seed(t + 3 * n + 7 * k)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()  # noqa: E731
    x, w = ints(t, k) * _powers(k, 4, 1), ints(n, k) * _powers(k, 3, 2) * _powers(n, 2, 1)[:, None]
    row = torch.exp2(torch.arange(t, device="cuda").float() % 5)[:, None]
    ref = (x @ w.t()) * row
    return (x * row).to(DT[dt]), w, ref


def _strided(x, pad, offset=0):
    big = torch.full((x.shape[0], x.shape[1] + pad + offset), float("nan"), dtype=x.dtype, device=x.device)
    big[:, offset:offset + x.shape[1]] = x
    return big[:, offset:offset + x.shape[1]]


def _splits(out_dt, t, n, k):
    """Ranges of k: with x quantised the workspace holds their partial sums alone, if there are several."""
    from bit_quantized_shampoo_amd import _lib as L
    code = {"f32": L.F32, "bf16": L.BF16, "f16": L.F16}[out_dt]
    return L.lib().shampoo4_fp8_linear_workspace_bytes(code, t, n, k, 1) // (4 * t * n)


def _check(t, n, k, out_dt):
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store, fp8_store_weight
    x, w, ref = _operands(t, n, k, out_dt)
    w8, x8 = fp8_store_weight(w), fp8_store(x)
    announce(f"exact fp8 linear {t}x{n}x{k} {out_dt}")
    want = ref.to(DT[out_dt])
    assert torch.equal(fp8_linear(x8, w8, dtype=DT[out_dt]), want)
    assert torch.equal(fp8_linear(_strided(x, 3, 1), w8), want)
    base = torch.randint(-50, 51, (t, n), device="cuda").float()
    for pad in (0, 5):
        out = torch.full((t, n + pad), 7.0, dtype=DT[out_dt], device="cuda")
        out[:, :n] = base.to(DT[out_dt])
        fp8_linear(x8, w8, out=out[:, :n], accumulate=True)
        assert torch.equal(out[:, :n], (ref + base).to(DT[out_dt])) and bool((out[:, n:] == 7).all())


@pytest.mark.parametrize("out_dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,n,k", [(1, 16, 128), (1, 1000, 4100), (7, 333, 700), (16, 520, 1024), (33, 200, 1300),
                                   (64, 130, 2000)])
def test_rows(t, n, k, out_dt):
    require_gpu()
    _check(t, n, k, out_dt)


@pytest.mark.parametrize("out_dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,n,k", [(64, 64, 2176), (65, 130, 900), (128, 192, 384), (300, 700, 1153), (777, 577, 1100)])
def test_tiles_of_64(t, n, k, out_dt):
    require_gpu()
    _check(t, n, k, out_dt)


@pytest.mark.parametrize("t,n,k,out_dt", [(2048, 2048, 256, "bf16"), (2000, 1100, 384, "bf16"), (4095, 4090, 300, "bf16"),
                                          (1990, 2041, 900, "f32"), (2048, 2048, 512, "f16")])
def test_tiles_of_128(t, n, k, out_dt):
    require_gpu()
    _check(t, n, k, out_dt)


@pytest.mark.parametrize("t,n,k", [(4096, 4096, 1152), (3841, 4000, 4000), (16384, 4096, 256), (12289, 5000, 1160)])
def test_tiles_of_256(t, n, k):
    """One tile a workgroup and several, whole and ragged, odd numbers of blocks of k among them."""
    require_gpu()
    _check(t, n, k, "bf16")


@pytest.mark.parametrize("t,n,k,out_dt", [
    (256, 300, 4100, "bf16"), (300, 300, 4096, "f32"), (700, 1000, 8200, "f32"),                   # 64 x 64
    (512, 4096, 14336, "bf16"), (500, 4090, 14300, "bf16"),                                         # 128 x 128
    (1024, 1024, 8192, "f32"), (1001, 1019, 8100, "f32"), (1000, 1020, 8192, "f16"),
    (768, 2816, 14336, "bf16"), (720, 2801, 14300, "bf16"), (2041, 4090, 14130, "bf16"),            # 256 x 256
    (1280, 3328, 32768, "bf16"), (1270, 3321, 32650, "bf16"),                                       # more than CUs
])
def test_ranges_of_k(t, n, k, out_dt):
    """Partial sums of ranges of k, joined: on every size of tile, whole and ragged; a last range of an odd number of
    blocks.  (Which tile is taken follows from estimated times; the comments say what it was when this was written.)"""
    require_gpu()
    if _splits(out_dt, t, n, k) < 2:
        pytest.skip("one range of k is taken here")
    _check(t, n, k, out_dt)


@pytest.mark.parametrize("t", [20, 70])
def test_longest_rows(t):
    """Rows of more than 2^23 columns are taken by the row kernel, however many there are.  Entries of x are 0 and
    +-1, one in 512, so sums stay below 2^15."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store, fp8_store_weight
    n, k = 35, (1 << 23) + 200
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.zeros((t, k), dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, k, (t, k // 512), generator=g, device="cuda")
    x.scatter_(1, at, (torch.randint(0, 2, at.shape, generator=g, device="cuda") * 2 - 1).bfloat16())
    x[:, -1] = 1
    w = torch.randint(-3, 4, (n, k), generator=g, device="cuda").bfloat16()
    ref = torch.zeros((t, n), device="cuda")
    for i in range(0, k, 1 << 20):
        ref += x[:, i:i + (1 << 20)].float() @ w[:, i:i + (1 << 20)].float().t()
    w8 = fp8_store_weight(w)
    announce(f"exact fp8 linear {t}x{n}x{k}")
    for out_dt in ("bf16", "f32"):
        want = ref.to(DT[out_dt])
        assert torch.equal(fp8_linear(x, w8, dtype=DT[out_dt]), want)
        assert torch.equal(fp8_linear(fp8_store(x), w8, dtype=DT[out_dt]), want)


@pytest.mark.parametrize("t,n,k,out_dt", [(3, 40, 300, "bf16"), (40, 40, 300, "f32"), (150, 70, 1100, "bf16"),
                                          (2304, 2304, 300, "bf16"), (4096, 4096, 1152, "bf16")])
def test_offsets_beyond_32_bits(t, n, k, out_dt):
    """x, and y at a distance of more than 2^31 elements from its first row, as columns of one long matrix."""
    require_gpu()
    from bit_quantized_shampoo_amd import fp8_linear, fp8_store_weight
    x, w, ref = _operands(t, n, k, out_dt)
    ld = (1 << 31) // (t - 1) * 9 // 8 + k + n + 9
    announce(f"exact fp8 linear {t}x{n}x{k} {out_dt}, rows {ld} apart")
    big = torch.empty((t, ld), dtype=DT[out_dt], device="cuda")
    big[:, :k] = x
    y = big[:, -n - 1:-1]
    big[:, -n - 2] = 7.0
    big[:, -1] = 7.0
    w8 = fp8_store_weight(w)
    fp8_linear(big[:, :k], w8, out=y)
    assert torch.equal(y, ref.to(DT[out_dt]))
    fp8_linear(big[:, :k], w8, out=y, accumulate=True)
    assert torch.equal(y, (ref.to(DT[out_dt]).float() + ref).to(DT[out_dt]))
    assert bool((big[:, -n - 2] == 7).all()) and bool((big[:, -1] == 7).all()) and torch.equal(big[:, :k], x)
