"""8-bit activation checkpoints, the activations that keep them and the weight gradient that
reads them, on the GPU against the float64 oracle.

Tolerances, with u the unit roundoff of the stored type (bf16 2^-8, f16 2^-11, f32 2^-24,
as a bound on one rounding to nearest relative to the result):
* codes, scales and restored values are exact;
* activations: z = the sigmoid's argument is rounded in fp32, so exp(-z) is off by a factor
  of up to 1 + |z| 2^-23, and a handful of fp32 operations follow: (|z| + 16) 2^-23 of the
  terms' sizes, plus u of the result for the store.  1 - sigmoid is off by 2^-24 of 1, which
  the derivative multiplies by |x dz|;
* weight gradient: products are exact, and a sum of T terms in fp32, in any order, is within
  T 2^-23 (one rounding or truncation each) of the sum of the terms' sizes."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


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


def _check_store(x):
    from bit_quantized_shampoo_amd import act8_load, act8_store
    t, c = x.shape
    a = act8_store(x)
    torch.cuda.synchronize()
    codes, scales = o.act8_store(_np(x))
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    ref = o.act8_load(codes, scales, t, c)
    for dt in DT.values():
        y = act8_load(a, dtype=dt)
        assert y.dtype == dt
        lim = 65504.0 if dt == torch.float16 else np.inf
        # float32 first: the restored value is exact in it, and in bfloat16
        want = torch.from_numpy(np.clip(ref, -lim, lim).astype(np.float32)).to(dt)
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    return a


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,c", [(1, 1), (1, 1024), (31, 7), (32, 16), (33, 129), (257, 640), (100, 1153)])
def test_store_is_exact(t, c, dt):
    require_gpu()
    rng = np.random.default_rng(t * 1000 + c)
    announce(f"act8 store {t}x{c} {dt}")
    x = _rand(rng, t, c, dt)
    a = _check_store(x)
    from bit_quantized_shampoo_amd import act8_load, act8_store
    b = act8_store(_strided(x, 5, 3))
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    out = torch.full((t, c + 9), 5.0, dtype=DT[dt], device="cuda")
    act8_load(a, out=out[:, 4:4 + c])
    assert torch.equal(out[:, 4:4 + c], act8_load(a, dtype=DT[dt]))
    assert bool((out[:, :4] == 5).all()) and bool((out[:, 4 + c:] == 5).all())


def test_store_special_values():
    """Zero blocks, subnormals, steps at the edges of the power-of-two rule and of rounding,
    the largest numbers, infinities and NaN in one column of many."""
    require_gpu()
    x = np.zeros((64, 48), np.float32)
    rng = np.random.default_rng(5)
    x[:, 1] = rng.standard_normal(64) * 1e-40                     # subnormal
    x[:, 2] = 2.0 ** -126
    x[3, 3], x[4, 3] = 127.0, 63.5                                # exactly 127 steps of 1, and a tie
    x[3, 4], x[4, 4] = np.nextafter(np.float32(127), np.float32(128)), 1.0
    x[:, 5] = np.arange(64) + 0.5                                 # ties in steps of 1
    x[0, 5] = 127.0
    x[:, 6] = np.float32(3.4e38)
    x[:, 7] = -np.finfo(np.float32).max
    x[:, 8] = rng.standard_normal(64)
    x[5, 8] = np.inf
    x[:, 9] = rng.standard_normal(64)
    x[40, 9] = np.nan
    x[:, 10] = rng.standard_normal(64) * 2.0 ** rng.integers(-20, 20, 64)
    x[:, 11] = 65504.0
    x[:, 12] = -0.0
    x[1, 13] = -1e-45
    for k in range(14, 48):
        x[:, k] = rng.standard_normal(64) * 2.0 ** (8 * (k - 30))
    announce("act8 store special values")
    a = _check_store(torch.from_numpy(x).cuda())
    assert int(a.scales[0, 8]) == 255 and int(a.scales[1, 8]) != 255
    assert int(a.scales[1, 9]) == 255 and int(a.scales[0, 9]) != 255
    _check_store(torch.from_numpy(x).cuda().bfloat16())


def test_store_offsets_beyond_32_bits():
    """A leading dimension that puts the last rows more than 2^31 elements in."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_store
    ld = (1 << 31) // 32 + 64
    announce("act8 store with 64-bit offsets")
    big = torch.zeros((40, ld), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(40, 50, device="cuda").bfloat16()
    big[:, -50:] = x
    a, b = act8_store(big[:, -50:]), act8_store(x)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,c", [(1, 5), (45, 300)])
def test_activation_matches_oracle(t, c, dt, gated, kind):
    require_gpu()
    from bit_quantized_shampoo_amd import act8_store, activation_backward, activation_forward
    rng = np.random.default_rng(7)
    announce(f"activation {kind} gated={gated} {t}x{c} {dt}")
    g = _strided(_rand(rng, t, c, dt, 2.0), 3, 1)
    u = _strided(_rand(rng, t, c, dt), 6) if gated else None
    h, g8, u8, h8 = activation_forward(g, u, kind=kind)
    x = _np(g)
    z, dz = o.act_argument(x, kind)
    up = _np(u) if gated else np.ones_like(x)
    ref = o.activation(x, kind) * up
    # 2^-149 is the underflow of exp and of the products, times the factors after it
    tol = np.abs(ref) * ((np.abs(z) + 16) * 2.0 ** -23 + U[dt]) + TINY[dt] + 2.0 ** -120 * np.abs(x * up)
    assert np.all(np.abs(_np(h) - ref) <= tol)
    for kept, src in ((g8, g), (u8, u), (h8, h)):
        if kept is not None:
            want = act8_store(src)
            assert torch.equal(kept.codes, want.codes) and torch.equal(kept.scales, want.scales)
    assert (u8 is not None) == gated
    # backward from the restored values
    dh = _rand(rng, t, c, dt)
    dg, du = activation_backward(dh, g8, u8, kind=kind)
    xg = o.act8_load(g8.codes.cpu().numpy(), g8.scales.cpu().numpy(), t, c)
    xu = o.act8_load(u8.codes.cpu().numpy(), u8.scales.cpu().numpy(), t, c) if gated else np.ones_like(xg)
    z, dz = o.act_argument(xg, kind)
    d = _np(dh)
    ref = d * xu * o.activation_derivative(xg, kind)
    sg = 1 / (1 + np.exp(-z))
    rel = (np.abs(z) + 16) * 2.0 ** -23
    size = np.abs(d * xu) * ((sg + np.abs(xg * sg * (1 - sg) * dz)) * rel + np.abs(xg * dz) * 2.0 ** -23)
    assert np.all(np.abs(_np(dg) - ref) <= size + U[dt] * np.abs(ref) + TINY[dt])
    if gated:
        ref = d * o.activation(xg, kind)
        assert np.all(np.abs(_np(du) - ref) <= np.abs(ref) * (rel + U[dt]) + TINY[dt])
    else:
        assert du is None
    # the gradient may take its input's place
    again, _ = activation_backward(dh, g8, u8, kind=kind, dgate=dh)
    assert again is dh and torch.equal(dh, dg)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_gradient_is_the_difference(kind):
    """dgate and dup against central differences of the float64 forward formula at the
    restored values: the difference's own error is about 1e-9, so fp32's decides (1e-5 of the
    factors' sizes covers (|z| + 16) 2^-23 for |z| up to 60)."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_store, activation_backward
    rng = np.random.default_rng(11)
    g8, u8 = act8_store(_rand(rng, 64, 40, "f32")), act8_store(_rand(rng, 64, 40, "f32"))
    g, u = _np(act8_load(g8, torch.float32)), _np(act8_load(u8, torch.float32))
    dh = _rand(rng, 64, 40, "f32")
    announce(f"activation differences {kind}")
    dg, du = activation_backward(dh, g8, u8, kind=kind)
    e = 1e-5
    diff = _np(dh) * u * (o.activation(g + e, kind) - o.activation(g - e, kind)) / (2 * e)
    size = np.abs(_np(dh) * u) * (1 + np.abs(g))
    assert np.all(np.abs(_np(dg) - diff) <= 1e-5 * size + 1e-12)
    diff = _np(dh) * o.activation(g, kind)
    assert np.all(np.abs(_np(du) - diff) <= 1e-5 * np.abs(diff) + 1e-12)


def test_activation_inference_form_and_extremes():
    """No checkpoints kept; very large arguments; an infinite or NaN activation is NaN or
    infinite where the formula is, and its block restores as NaN."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, activation_forward
    x = torch.tensor([[-1e30, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e30, float("inf"), float("nan")]],
                     device="cuda")
    for kind in ("silu", "gelu"):
        announce(f"activation extremes {kind}")
        h, g8, u8, h8 = activation_forward(x, kind=kind, checkpoint=False, save_output=False)
        assert g8 is None and u8 is None and h8 is None
        h = _np(h)[0]
        assert np.all(np.abs(h[:4]) < 1e-7) and h[4] == 0
        assert np.allclose(h[5:9], [20.0, 90.0, 200.0, 1e30], rtol=1e-6) and np.isinf(h[9]) and np.isnan(h[10])
        _, g8, _, _ = activation_forward(x, kind=kind)
        y = _np(act8_load(g8))[0]
        assert np.isnan(y[9]) and np.isnan(y[10]) and np.all(np.isfinite(y[:9]))


def test_activation_empty():
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_weight_grad, activation_backward, activation_forward
    x = torch.empty(0, 12, device="cuda")
    h, g8, u8, h8 = activation_forward(x, x)
    assert h.shape == (0, 12) and act8_load(h8).shape == (0, 12)
    dg, du = activation_backward(h, g8, u8)
    assert dg.shape == du.shape == (0, 12)
    g = torch.ones(5, 12, device="cuda")
    announce("weight gradient over no rows")
    act8_weight_grad(torch.empty(0, 5, device="cuda"), h8, out=g, beta=0.5)
    assert bool((g == 0.5).all())
    assert bool((act8_weight_grad(torch.empty(0, 5, device="cuda"), h8) == 0).all())


def _wgrad_case(t, n, c, dt, seed, alpha=1.0, beta=0.0, pad=0):
    from bit_quantized_shampoo_amd import act8_store, act8_weight_grad
    rng = np.random.default_rng(seed)
    x8 = act8_store(_rand(rng, t, c, "f32"))
    dy = _rand(rng, t, n, dt, 1e-2)
    if pad:
        dy = _strided(dy, pad, 1)
    g0 = torch.from_numpy(rng.standard_normal((n, c + pad)).astype(np.float32)).cuda()
    out = g0.clone()
    announce(f"weight gradient T={t} N={n} C={c} {dt} alpha={alpha} beta={beta} pad={pad}")
    act8_weight_grad(dy, x8, out=out[:, :c], alpha=alpha, beta=beta)
    torch.cuda.synchronize()
    x = o.act8_load(x8.codes.cpu().numpy(), x8.scales.cpu().numpy(), t, c)
    d = _np(dy)
    ref = alpha * (d.T @ x) + beta * _np(g0)[:, :c]
    size = abs(alpha) * (np.abs(d).T @ np.abs(x)) + abs(beta) * np.abs(_np(g0)[:, :c])
    err = np.abs(_np(out)[:, :c] - ref)
    assert np.all(err <= (t + 4) * 2.0 ** -23 * size + 1e-37)
    # rounding errors of a long sum do not line up: far below the bound in the mean
    assert np.linalg.norm(err) <= 4e-6 * np.linalg.norm(size)
    assert torch.equal(out[:, c:], g0[:, c:])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,n,c", [(1, 1, 1), (32, 128, 128), (33, 130, 17), (100, 64, 333), (1000, 257, 96),
                                   (2049, 300, 260)])
def test_weight_grad(t, n, c, dt):
    require_gpu()
    _wgrad_case(t, n, c, dt, seed=t + n + c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_weight_grad_accumulates_into_a_view(dt):
    require_gpu()
    _wgrad_case(300, 150, 77, dt, seed=3, alpha=0.5, beta=1.0, pad=5)
    _wgrad_case(5000, 70, 131, dt, seed=4, alpha=-2.0, beta=0.25, pad=3)


@pytest.mark.parametrize("n,c", [(70, 131), (64, 131), (1, 7), (5, 260)])
def test_weight_grad_joins_row_ranges_of_contiguous_outputs(n, c):
    require_gpu()
    _wgrad_case(2000, n, c, "f32", seed=n + c, alpha=1.5, beta=-0.5)
    _wgrad_case(4000, n, c, "bf16", seed=n + c + 1)


def test_weight_grad_large_and_deterministic():
    """A layer of the transformer shapes: against float64 on the GPU, twice the same bits, and
    beta = 0 reads nothing of a NaN-filled output."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_store, act8_weight_grad
    g = torch.Generator(device="cuda").manual_seed(1)
    t, n, c = 4100, 1024, 4096
    x8 = act8_store(torch.randn(t, c, generator=g, device="cuda"))
    dy = torch.randn(t, n, generator=g, device="cuda").bfloat16()
    announce("weight gradient 4100 x 1024 x 4096")
    out = torch.full((n, c), float("nan"), device="cuda")
    act8_weight_grad(dy, x8, out=out)
    assert torch.equal(out, act8_weight_grad(dy, x8))
    x = act8_load(x8, torch.float32).double()
    ref = dy.double().t().contiguous() @ x
    assert float((out.double() - ref).norm() / ref.norm()) <= 2e-6


def test_weight_grad_non_finite():
    """An infinite gradient stays infinite in its row of G (or NaN where the other factor is
    0), a non-finite activation makes its column NaN, everything else is untouched."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_store, act8_weight_grad
    x = torch.ones(64, 40, device="cuda")
    x[10, 7] = float("nan")
    x8 = act8_store(x)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        dy = torch.ones(64, 20, device="cuda", dtype=dt)
        dy[3, 5] = float("inf")
        announce(f"weight gradient non-finite {dt}")
        g = act8_weight_grad(dy, x8).cpu()
        assert bool(torch.isnan(g[:, 7]).all())
        keep = torch.arange(40) != 7
        assert bool(torch.isinf(g[5, keep]).all())
        rows = torch.arange(20) != 5
        assert bool((g[rows][:, keep] == 64).all())


def test_other_stream():
    """Work on a stream of its own, ordered by the caller."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_store
    x = torch.randn(3000, 700, device="cuda").bfloat16()
    want = act8_load(act8_store(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    announce("act8 on another stream")
    y = act8_load(act8_store(x, stream=s), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)


def test_weight_grad_with_a_very_long_leading_dimension():
    """A leading dimension of more than 2^24 elements, and rows more than 2^31 bytes apart in all."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_store, act8_weight_grad
    t, n, c = 70, 130, 40
    announce("weight gradient, leading dimension 2^24 + 8")
    big = torch.zeros((t, (1 << 24) + 8), dtype=torch.bfloat16, device="cuda")
    dy = torch.randn(t, n, device="cuda").bfloat16()
    big[:, 5:5 + n] = dy
    x8 = act8_store(torch.randn(t, c, device="cuda"))
    assert torch.equal(act8_weight_grad(big[:, 5:5 + n], x8), act8_weight_grad(dy, x8))


def test_weight_grad_ignores_what_lies_between_rows():
    """NaN in the padding of dY's rows, and in what follows its last row, changes nothing."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_store, act8_weight_grad
    for t, n, c in ((300, 130, 200), (64, 300, 270)):
        for dt in (torch.bfloat16, torch.float32):
            dy = torch.randn(t, n, device="cuda").to(dt)
            big = torch.full((t + 9, n + 37), float("nan"), dtype=dt, device="cuda")
            big[:t, :n] = dy
            x8 = act8_store(torch.randn(t, c, device="cuda"))
            announce(f"weight gradient between rows {t}x{n}x{c} {dt}")
            assert torch.equal(act8_weight_grad(big[:t, :n], x8), act8_weight_grad(dy, x8))


def test_binding_refusals():
    require_gpu()
    import bit_quantized_shampoo_amd as s4
    x = torch.randn(64, 48, device="cuda")
    x8 = s4.act8_store(x)
    bad = [
        (ValueError, lambda: s4.act8_store(x.t())),                                  # column-major
        (ValueError, lambda: s4.act8_store(x[:, ::2])),
        (ValueError, lambda: s4.act8_store(x[:1].expand(64, 48))),                   # broadcast rows
        (ValueError, lambda: s4.act8_store(x[0])),
        (ValueError, lambda: s4.act8_store(x[:, :0])),
        (TypeError, lambda: s4.act8_store(x.double())),
        (ValueError, lambda: s4.act8_store(x[:32], out=x8)),
        (ValueError, lambda: s4.Act8(x8.codes, x8.scales, 64, 49)),
        (ValueError, lambda: s4.Act8(x8.codes.view(torch.uint8), x8.scales, 64, 48)),
        (TypeError, lambda: s4.act8_load(x8, dtype=torch.int8)),
        (ValueError, lambda: s4.act8_load(x8, out=x[:63])),
        (ValueError, lambda: s4.activation_forward(x, x[:32])),
        (TypeError, lambda: s4.activation_forward(x, x.bfloat16())),
        (ValueError, lambda: s4.activation_backward(x[:32], x8)),
        (ValueError, lambda: s4.activation_backward(x, x8, dup=x)),
        (TypeError, lambda: s4.act8_weight_grad(x, x)),
        (ValueError, lambda: s4.act8_weight_grad(x[:32], x8)),
        (ValueError, lambda: s4.act8_weight_grad(x, x8, beta=1.0)),
        (TypeError, lambda: s4.act8_weight_grad(x, x8, out=torch.zeros(48, 48, device="cuda").bfloat16())),
        (ValueError, lambda: s4.embedding(x, torch.zeros(2, 2, dtype=torch.int64, device="cuda"))),
        (TypeError, lambda: s4.embedding(x, torch.zeros(2, device="cuda"))),
        (ValueError, lambda: s4.embedding_grad(x, torch.zeros(3, dtype=torch.int64, device="cuda"), 5)),
        (ValueError, lambda: s4.embedding_grad(x, torch.zeros(64, dtype=torch.int64, device="cuda"), 5, accumulate=True)),
        (ValueError, lambda: s4.embedding_grad(x, torch.zeros(64, dtype=torch.int64, device="cuda"), 5,
                                               workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: s4.token_logprobs(x, torch.zeros(63, dtype=torch.int64, device="cuda"))),
        (ValueError, lambda: s4.policy_loss(x, torch.zeros(64, dtype=torch.int64, device="cuda"), x[:, 0].contiguous(),
                                            x[:, 0].contiguous(), x[:, 0].contiguous(), kl_coef=0.1)),
        (ValueError, lambda: s4.policy_loss(x, torch.zeros(64, dtype=torch.int64, device="cuda"), x[:, 0],
                                            x[:, 0].contiguous(), x[:, 0].contiguous())),
        (s4.Shampoo4Error, lambda: s4.policy_loss(x, torch.zeros(64, dtype=torch.int64, device="cuda"),
                                                  *[x[:, 0].contiguous()] * 3, clip_low=-1.0)),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {k} was not refused")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_gradient_at_extremes(kind):
    """Far from 0 the derivative is 0 or 1, also where the cube of the argument overflows."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_store, activation_backward
    x = torch.tensor([[-1e30, -1e20, -1e10, -300.0, 300.0, 1e10, 1e20, 1e30]], device="cuda")
    announce(f"activation gradient extremes {kind}")
    dg, _ = activation_backward(torch.full_like(x, 2.0), act8_store(x), kind=kind)
    assert torch.equal(dg.abs(), torch.tensor([[0.0] * 4 + [2.0] * 4], device="cuda"))


def test_captured_graphs():
    """Forward, backward and weight gradient (with row ranges to join) from a captured graph,
    replayed with other work between the replays, against the eager results."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_store, act8_weight_grad, activation_backward, activation_forward
    g, u, dh = (torch.randn(2100, 300, device="cuda").bfloat16() for _ in range(3))

    def call():
        h, g8, u8, h8 = activation_forward(g, u)
        dg, du = activation_backward(dh, g8, u8)
        return h, dg, du, act8_weight_grad(dh, h8), act8_load(act8_store(h))

    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    announce("activation and weight gradient graph")
    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        torch.randn(1000, 1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_keeps_its_small_values(kind):
    """Where the sigmoid is below fp32's normal range (z from -87.3 down to -103.3) it is held as a subnormal number,
    half a step of 2^-149 from its value: the products with x and with a large factor are what the formula gives.
    z itself is within 5 roundings of its value for GELU, so exp(z) is within 3 |z| 2^-23."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, activation_backward, activation_forward
    x = np.linspace(-110.0, -84.0, 208) if kind == "silu" else np.linspace(-11.2, -9.6, 208)
    g = torch.from_numpy(np.tile(x.astype(np.float32), (32, 1))).cuda()
    for up in (1.0, 1e20):
        announce(f"activation of small values {kind} up={up}")
        u = torch.full_like(g, up)
        h, g8, u8, _ = activation_forward(g, u, kind=kind)
        xs = _np(g)
        z, _ = o.act_argument(xs, kind)
        ref = o.activation(xs, kind) * up
        tol = np.abs(ref) * (3 * np.abs(z) + 16) * 2.0 ** -23 + 2.0 ** -149 * (np.abs(xs) + 1) * max(up, 1.0)
        assert np.all(np.abs(_np(h) - ref) <= tol)
        dh = torch.full_like(g, 1e15)
        dg, du = activation_backward(dh, g8, u8, kind=kind)
        xs, xu = _np(act8_load(g8, torch.float32)), _np(act8_load(u8, torch.float32))
        z, dz = o.act_argument(xs, kind)
        rel = (3 * np.abs(z) + 16) * 2.0 ** -23
        ref = o.activation(xs, kind) * 1e15
        assert np.all(np.abs(_np(du) - ref) <= np.abs(ref) * rel + 2.0 ** -149 * (np.abs(xs) + 1) * 1e15)
        ref = o.activation_derivative(xs, kind) * xu * 1e15
        assert np.all(np.abs(_np(dg) - ref) <= np.abs(ref) * 2 * rel + 2.0 ** -149 * (np.abs(xs * dz) + 2) * xu * 1e15)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_gradient_keeps_its_last_bits(kind):
    """For z in 10 .. 25 the derivative is 1 and a small term x (1 - sg) z' of it: the sigmoid's sum, its reciprocal
    and the two last roundings are within 2^-24 each, and the term, 0.3% at most, adds (3 |z| 2^-23) of itself: 6 2^-24
    of dh in all.  1 - sg taken as a difference would lose 2^-24 times x z' (15 to 60) more."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_store, activation_backward
    lo, hi = (10.0, 25.0) if kind == "silu" else (4.2, 6.3)
    rng = np.random.default_rng(2)
    # columns of several scales: each block's largest value is in one of them
    x = rng.uniform(lo, hi, (64, 300)).astype(np.float32)
    g8 = act8_store(torch.from_numpy(x).cuda())
    xs = _np(act8_load(g8, torch.float32))
    dh = torch.from_numpy(rng.standard_normal((64, 300)).astype(np.float32)).cuda()
    announce(f"activation gradient's last bits {kind}")
    dg, _ = activation_backward(dh, g8, kind=kind)
    d = _np(dh)
    ref = d * o.activation_derivative(xs, kind)
    z, _ = o.act_argument(xs, kind)
    on = (z >= 10) & (z <= 25)
    assert on.mean() > 0.8
    assert np.all((np.abs(_np(dg) - ref) <= 6 * 2.0 ** -24 * np.abs(d))[on])


def test_weight_grad_of_half_a_billion_columns():
    """An output of 2^22 tiles, as wide as one launch takes with two rows: every product is exact."""
    require_gpu()
    from bit_quantized_shampoo_amd import act8_load, act8_store, act8_weight_grad
    c = (1 << 29) + 16
    announce("weight gradient 1 x 2 x (2^29 + 16)")
    x8 = act8_store((torch.arange(c, dtype=torch.int32, device="cuda") % 61 - 30).to(torch.bfloat16).view(1, c))
    g = act8_weight_grad(torch.tensor([[2.0, -1.0]], device="cuda").bfloat16(), x8)
    x = act8_load(x8, torch.float32)[0]
    assert torch.equal(g[1], -x) and torch.equal(g[0], x + x)
    assert float(x[c - 1]) == (c - 1) % 61 - 30
