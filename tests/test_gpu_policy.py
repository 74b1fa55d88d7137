"""The clipped policy loss with a KL term and the token log-probabilities, against the float64
oracle.

Bounds.  A row's sum of exponentials is a sum in fp32 whose longest chain is a thread's (up to
129 terms) and the joins after it, each term within 2^-22 (argument and exp2): relative
(129 + 40) 2^-24 + 2^-22 < 1.1e-5, so |logp error| <= 2e-5 + 2^-21 |logp|.  The ratio and exp(d)
carry that as a relative error: 1e-4 of the coefficient's terms covers it with its products.
A gradient's element adds the rounding u of its type (and f16's smallest step)."""

import numpy as np
import pytest
import torch

from oracle import train as o
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
CLIP = dict(clip_low=0.2, clip_high=0.28)


def _np(t):
    return t.detach().double().cpu().numpy()


def _case(rows, vocab, dt, seed=0, pad=0):
    rng = np.random.default_rng(seed + rows * 7 + vocab)
    z = torch.from_numpy((2 * rng.standard_normal((rows, vocab + pad))).astype(np.float32)).cuda().to(DT[dt])
    z = z[:, pad // 2:pad // 2 + vocab]
    y = rng.integers(0, vocab, rows)
    lp = o.log_softmax(_np(z))[np.arange(rows), y] if rows else np.zeros(0)
    c = {"z": z, "y": y, "old": lp + 0.3 * rng.standard_normal(rows), "ref": lp + 0.4 * rng.standard_normal(rows),
         "adv": rng.standard_normal(rows), "w": rng.random(rows) / max(rows, 1)}
    return {k: (v.astype(np.float32) if k in ("old", "ref", "adv", "w") else v) for k, v in c.items()}


def _run(c, kl, idt=torch.int64, **kw):
    from bit_quantized_shampoo_amd import policy_loss
    dev = {k: torch.from_numpy(c[k]).cuda() for k in ("old", "ref", "adv", "w")}
    return policy_loss(c["z"], torch.from_numpy(c["y"]).to(idt).cuda(), dev["old"], dev["adv"], dev["w"],
                       ref_logp=dev["ref"] if kl else None, kl_coef=kl, **CLIP, **kw)


def _check(c, kl, dt, got, gs=1.0):
    loss, logp, dz = got
    ref = o.policy(_np(c["z"]), c["y"], c["old"], c["adv"], c["w"], c["ref"], kl=kl, **CLIP)
    assert abs(float(loss) - ref[0]) <= 1e-4 * ref[3].sum() + 1e-30
    assert np.all(np.abs(_np(logp) - ref[1]) <= 2e-5 + 2.0 ** -21 * np.abs(ref[1]))
    if dz is not None:
        p = np.exp(o.log_softmax(_np(c["z"])))
        hot = np.zeros_like(p)
        on = (c["y"] >= 0) & (c["y"] < p.shape[1])
        hot[np.arange(len(p))[on], c["y"][on]] = 1
        # a ratio at an end of the clip range may fall on either side of it: then the whole term
        tol = gs * ref[3][:, None] * 1e-4 * (p + hot)
        assert np.all(np.abs(_np(dz) - gs * ref[2]) <= tol + U[dt] * np.abs(gs * ref[2]) + (2.0 ** -25 if dt == "f16" else 1e-37))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 5), (2, 64), (5, 1000), (70, 2051), (3, 9001), (70, 9001), (66, 20001),
                                        (2, 40961), (65, 65536), (1, 131071)])
def test_policy_loss(rows, vocab, dt):
    require_gpu()
    c = _case(rows, vocab, dt)
    announce(f"policy loss {rows}x{vocab} {dt}")
    _check(c, 0.05, dt, _run(c, 0.05))


@pytest.mark.parametrize("rows,vocab,dt", [(64, 70001, "f32"), (66, 131072, "bf16"), (64, 131104, "f16")])
def test_policy_loss_longest_rows(rows, vocab, dt):
    """The longest rows a workgroup holds, and rows it does not, with many rows."""
    require_gpu()
    c = _case(rows, vocab, dt)
    announce(f"policy loss {rows}x{vocab} {dt}")
    _check(c, 0.0, dt, _run(c, 0.0))


@pytest.mark.parametrize("rows,vocab", [(9, 301), (7, 30001)])
def test_policy_loss_strided_in_place_scaled(rows, vocab):
    require_gpu()
    c = _case(rows, vocab, "bf16", pad=7)
    announce(f"policy loss strided {rows}x{vocab}")
    loss, logp, dz = _run(c, 0.1, torch.int32, grad_scale=8.0)
    _check(c, 0.1, "bf16", (loss, logp, dz), gs=8.0)
    l1, p1, none = _run(c, 0.1, grad=False)
    assert none is None and torch.equal(l1, loss) and torch.equal(p1, logp)
    z = c["z"]
    l2, p2, d2 = _run(c, 0.1, grad_scale=8.0, dlogits=z)
    assert d2 is z and torch.equal(z, dz) and torch.equal(l2, loss) and torch.equal(p2, logp)


@pytest.mark.parametrize("vocab", [77, 20000])
@pytest.mark.parametrize("rows", [6, 100])
def test_rows_that_do_not_count(rows, vocab):
    """Weight 0 and targets outside the vocabulary: whatever the row holds, its gradient and
    log-probability are 0 and it adds nothing."""
    require_gpu()
    c = _case(rows, vocab, "f32")
    c["w"][1] = 0
    c["z"][1] = float("nan")
    c["old"][1] = c["adv"][1] = np.nan
    c["y"][2] = -1
    c["y"][3] = vocab
    c["w"][4] = 0
    c["z"][4] = float("-inf")
    c["ref"][4] = np.inf
    announce(f"policy masked rows {rows}x{vocab}")
    dz = torch.full((rows, vocab), float("nan"), device="cuda")
    loss, logp, dz = _run(c, 0.1, dlogits=dz)
    for t in (1, 2, 3, 4):
        assert float(logp[t]) == 0 and bool((dz[t] == 0).all())
    keep = [t for t in range(rows) if t not in (1, 2, 3, 4)]
    sub = {k: (v[torch.tensor(keep).cuda()] if k == "z" else v[keep]) for k, v in c.items()}
    _check(sub, 0.1, "f32", (loss, logp[keep], dz[keep]))
    c["w"][:] = 0
    loss, logp, dz = _run(c, 0.1)
    assert float(loss) == 0 and bool((dz == 0).all()) and bool((logp == 0).all())


@pytest.mark.parametrize("rows,vocab", [(4, 500), (70, 500), (4, 30000), (70, 30000)])
def test_masked_logits(rows, vocab):
    """Most of the vocabulary at -infinity (or the type's lowest value): probability 0, the
    same loss as over the rest; one row keeps a single word."""
    require_gpu()
    for low in (float("-inf"), torch.finfo(torch.float32).min):
        c = _case(rows, vocab, "f32")
        allowed = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        allowed[::37] = True
        c["y"] = (c["y"] // 37) * 37
        c["z"].masked_fill_(~allowed, low)
        c["z"][0] = low
        c["z"][0, c["y"][0]] = 1.0
        lp = o.log_softmax(_np(c["z"]))[np.arange(rows), c["y"]]
        c["old"], c["ref"] = (lp - 0.1).astype(np.float32), (lp + 0.2).astype(np.float32)
        announce(f"policy masked logits {rows}x{vocab} {low}")
        got = _run(c, 0.05)
        _check(c, 0.05, "f32", got)
        assert bool((got[2][:, ~allowed] == 0).all()) and abs(float(got[1][0])) <= 1e-6


def test_nan_and_infinite_logits_show():
    """A NaN or +infinity among a counted row's logits makes that row NaN, and no other."""
    require_gpu()
    for vocab in (300, 30000):
        c = _case(5, vocab, "f32")
        c["z"][1, 17] = float("nan")
        c["z"][3, vocab - 1] = float("inf")
        announce(f"policy non-finite {vocab}")
        loss, logp, dz = _run(c, 0.05)
        assert np.isnan(float(loss))
        bad = torch.tensor([False, True, False, True, False], device="cuda")
        assert torch.equal(torch.isnan(logp), bad)
        assert bool(torch.isnan(dz[bad]).any(1).all()) and bool(torch.isfinite(dz[~bad]).all())


def test_gradient_is_the_difference_of_the_loss():
    """dZ against central differences of the float64 loss: fp32's 1e-4 of the coefficient's
    terms, and 1e-8 for the difference."""
    require_gpu()
    c = _case(6, 9, "f32")
    # ratios inside and beyond the clip range, none at its ends
    lp = o.log_softmax(_np(c["z"]))[np.arange(6), c["y"]]
    c["old"] = (lp - np.log([0.5, 0.9, 1.05, 1.1, 1.6, 1.4])).astype(np.float32)
    announce("policy differences")
    _, _, dz = _run(c, 0.1)
    z, args = _np(c["z"]), (c["y"], c["old"], c["adv"], c["w"], c["ref"], 0.2, 0.28, 0.1)
    size = o.policy(z, *args)[3]
    for t in range(6):
        for v in range(9):
            zp, zm = z.copy(), z.copy()
            zp[t, v] += 1e-6
            zm[t, v] -= 1e-6
            diff = (o.policy(zp, *args)[0] - o.policy(zm, *args)[0]) / 2e-6
            assert abs(float(dz[t, v]) - diff) <= 1e-4 * size[t] + 1e-8


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(0, 50), (1, 131072), (3, 17), (65, 5000), (2, 300000), (70, 140000)])
def test_token_logprobs(rows, vocab, dt):
    require_gpu()
    from bit_quantized_shampoo_amd import token_logprobs
    c = _case(rows, vocab, dt)
    if rows > 2:
        c["y"][1] = -1
    announce(f"token logprobs {rows}x{vocab} {dt}")
    got = _np(token_logprobs(c["z"], torch.from_numpy(c["y"]).cuda()))
    if rows == 0:
        assert got.shape == (0,)
        return
    ref = o.log_softmax(_np(c["z"]))[np.arange(rows), np.maximum(c["y"], 0)]
    if rows > 2:
        ref[1] = 0
    assert np.all(np.abs(got - ref) <= 2e-5 + 2.0 ** -21 * np.abs(ref))


def test_no_rows():
    require_gpu()
    c = _case(0, 10, "bf16")
    loss, logp, dz = _run(c, 0.0)
    assert float(loss) == 0 and logp.shape == (0,) and dz.shape == (0, 10)


def test_deterministic_and_captured():
    """Twice the same bits, and the same from a captured graph over several replays with other
    work between them."""
    require_gpu()
    from bit_quantized_shampoo_amd import policy_loss
    for rows, vocab in ((8, 30000), (80, 3000)):
        c = _case(rows, vocab, "bf16")
        d = {k: torch.from_numpy(c[k]).cuda() for k in ("old", "ref", "adv", "w")}
        y = torch.from_numpy(c["y"]).cuda()
        call = lambda: policy_loss(c["z"], y, d["old"], d["adv"], d["w"], ref_logp=d["ref"], kl_coef=0.1)  # noqa: E731
        want = call()
        again = call()
        assert all(torch.equal(a, b) for a, b in zip(want, again))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        announce(f"policy graph {rows}x{vocab}")
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


def test_offsets_beyond_32_bits():
    """More than 2^31 logits; only the last rows count."""
    require_gpu()
    from bit_quantized_shampoo_amd import policy_loss
    rows, vocab = 33000, 65600
    announce("policy loss with 64-bit offsets")
    z = torch.empty((rows, vocab), dtype=torch.bfloat16, device="cuda")
    z[-70:] = torch.randn(70, vocab, device="cuda").bfloat16()
    y = torch.randint(0, vocab, (rows,), device="cuda")
    old, adv, w = torch.full((rows,), -11.0, device="cuda"), torch.randn(rows, device="cuda"), torch.zeros(rows, device="cuda")
    w[-70:] = 1.0
    want = policy_loss(z[-70:].clone(), y[-70:], old[-70:], adv[-70:], w[-70:])
    loss, logp, dz = policy_loss(z, y, old, adv, w, dlogits=z)
    assert torch.equal(dz[-70:], want[2]) and torch.equal(logp[-70:], want[1])
    assert abs(float(loss) - float(want[0])) <= 1e-5 * float(adv[-70:].abs().sum())
    assert bool((dz[-71] == 0).all()) and bool((dz[0] == 0).all()) and float(logp[:-70].abs().sum()) == 0


def _masked_rows(rows, vocab, dt, low):
    """Rows with finite masks of one size: words allowed in one place only, a masked tail, nothing but the mask, a
    maximum of the mask's size above ordinary logits, and every 37th word allowed."""
    c = _case(rows, vocab, dt)
    z, y = c["z"], c["y"]
    z[0, 20:] = low
    y[0] = 7
    z[1, vocab // 3:] = low
    y[1] = vocab // 3 - 1
    z[2] = low
    z[3, vocab // 2] = -low
    y[3] = vocab // 2
    for t in range(4, rows):
        z[t].masked_fill_(torch.arange(vocab, device="cuda") % 37 != 0, low)
        y[t] = y[t] // 37 * 37
    lp = o.log_softmax(_np(z))[np.arange(rows), y]
    c["old"], c["ref"] = (lp - 0.1).astype(np.float32), (lp + 0.2).astype(np.float32)
    return c


MASKS = (-1e4, -1e9, -5e9, -1e10, -1e12, -1e15, -1e20, -1e30, -1e38, "lowest")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(4, 500), (70, 3001), (5, 30000), (66, 70001)])
def test_finite_masks_of_any_size(rows, vocab, dt):
    """A finite logit is a logit: masks of every size have the probability that the definition gives them (0 beside
    ordinary logits, 1 / vocab in a row of nothing else).  The bounds are those of ordinary logits: differences to
    the maximum carry |z - m| 2^-23, which the terms' own size exp(z - m) outweighs (x exp(-x) < 0.4)."""
    require_gpu()
    from bit_quantized_shampoo_amd import token_logprobs
    for low in MASKS:
        low = torch.finfo(DT[dt]).min if low == "lowest" else low
        c = _masked_rows(rows, vocab, dt, low)
        announce(f"policy finite masks {rows}x{vocab} {dt} {low}")
        got = _run(c, 0.05)
        _check(c, 0.05, dt, got)
        assert abs(float(got[1][2]) + np.log(vocab)) <= 2e-5 + 2.0 ** -21 * np.log(vocab)
        # the rows' log-probabilities alone, also of a masked word and below a large maximum
        y = c["y"].copy()
        y[0], y[3] = vocab - 1, 1
        lp = o.log_softmax(_np(c["z"]))[np.arange(rows), y]
        got = _np(token_logprobs(c["z"], torch.from_numpy(y).cuda()))
        assert np.all(np.abs(got - lp) <= 2e-5 + 2.0 ** -21 * np.abs(lp))


KL_STEPS = (0.0, 1e-5, -1e-5, 1e-4, -1e-4, 1e-3, -1e-3, 1e-2, -1e-2, 0.1, -0.1, 0.3, -0.4, 0.49, -0.51, 0.7, 2.0, -3.0)


@pytest.mark.parametrize("vocab", [5, 30000])
def test_kl_term_near_the_reference(vocab):
    """The KL term and its derivative are relative to themselves: exp(d) - d - 1 and 1 - exp(d) lose nothing where d
    is near 0.  d is exact in fp32 for ref within a factor of 2 of logp; then a dozen roundings of a series, or an
    expm1 within 2^-22 of at most 3.7 times the term: 2^-18 of the term covers both.  With A = 0 the gradient's
    coefficient is the KL term's derivative alone; where rows are split it is taken at a log-probability joined in
    another order, 2^-21 of it away from the one returned."""
    require_gpu()
    from bit_quantized_shampoo_amd import policy_loss
    rows, kl = len(KL_STEPS), 0.04
    c = _case(rows, vocab, "f32")
    y = torch.from_numpy(c["y"]).cuda()
    zero, old = torch.zeros(rows, device="cuda"), torch.from_numpy(c["old"]).cuda()
    one = torch.ones(rows, device="cuda")
    announce(f"policy KL near the reference {vocab}")
    logp = policy_loss(c["z"], y, old, zero, one, grad=False)[1]
    ref = logp + torch.tensor(KL_STEPS, device="cuda")
    _, again, dz = policy_loss(c["z"], y, old, zero, one, ref_logp=ref, kl_coef=kl)
    assert torch.equal(again, logp)
    d = _np(ref) - _np(logp)
    coef = -kl * np.expm1(d)
    moved = kl * np.exp(d) * 2.0 ** -21 * np.abs(_np(logp)) if vocab > 9000 else np.zeros(rows)
    p = np.exp(o.log_softmax(_np(c["z"])))
    hot = np.zeros_like(p)
    hot[np.arange(rows), c["y"]] = 1
    assert np.all(np.abs(_np(dz) - coef[:, None] * (hot - p)) <= (2.0 ** -18 * np.abs(coef) + moved)[:, None] * (p + hot) + 1e-37)
    for t in range(rows):
        # expm1(d) - d in float64, by its series where that is short
        x = d[t]
        k = x * x / 2 * (1 + x / 3 * (1 + x / 4 * (1 + x / 5))) if abs(x) < 1e-3 else np.expm1(x) - x
        w = zero.clone()
        w[t] = 1
        loss = float(policy_loss(c["z"], y, old, zero, w, ref_logp=ref, kl_coef=kl, grad=False)[0])
        assert abs(loss - kl * k) <= 2.0 ** -18 * kl * k and loss >= 0


@pytest.mark.parametrize("vocab", [5, 30000])
def test_ratio_that_overflows(vocab):
    """exp(logp - old) beyond fp32: without an advantage it counts for nothing, with a positive one it is clipped."""
    require_gpu()
    c = _case(4, vocab, "f32")
    c["old"] = (c["old"] - 200).astype(np.float32)
    c["adv"] = np.array([0.0, 1.5, -0.0, 0.5], np.float32)
    announce(f"policy ratio overflow {vocab}")
    loss, _, dz = _run(c, 0.0)
    want = -1.28 * float((c["w"].astype(np.float64) * c["adv"]).sum())
    assert abs(float(loss) - want) <= 1e-6 * abs(want)
    assert bool((dz == 0).all())
