"""Host-only checks of the training operators: the library exports what its header declares,
every call refuses what the header says it refuses before anything reaches a device, the
binding checks its arguments, and the oracle's gradients agree with differences of its own
forward formulas."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from bit_quantized_shampoo_amd import _lib as L
from bit_quantized_shampoo_amd import train as T
from oracle import train as o

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "shampoo4_train.h")
P = 0x10000          # an aligned address that no refused call may touch


def _lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return L.lib()


def test_header_declares_the_binding_surface():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"SHAMPOO4_API[^;(]*?\b(shampoo4_\w+)\s*\(", text)))
    assert declared == sorted(L.EXPORTED_TRAIN)
    lib = _lib()
    for name in declared:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("rows,cols,status,codes", [
    (1, 1, L.OK, 32 * 16), (0, 5, L.OK, 0), (33, 17, L.OK, 64 * 32), (-1, 4, L.ESHAPE, 0), (4, 0, L.ESHAPE, 0),
    (1 << 31, 4, L.ESHAPE, 0),
])
def test_act8_bytes(rows, cols, status, codes):
    c, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert _lib().shampoo4_act8_bytes(rows, cols, ctypes.byref(c), ctypes.byref(s)) == status
    if status == L.OK:
        assert (c.value, s.value) == (codes, codes // 32)


def test_act8_refusals():
    lib = _lib()
    store = lib.shampoo4_act8_store
    assert store(3, 4, 4, P, 4, P, P, None) == L.EINVAL              # element type
    assert store(L.F32, -1, 4, P, 4, P, P, None) == L.ESHAPE
    assert store(L.F32, 4, 0, P, 4, P, P, None) == L.ESHAPE
    assert store(L.F32, 4, 4, P, 3, P, P, None) == L.ESHAPE          # leading dimension
    assert store(L.F32, 4, 4, None, 4, P, P, None) == L.EINVAL
    assert store(L.F32, 4, 4, P, 4, None, P, None) == L.EINVAL
    assert store(L.F32, 4, 4, P, 4, P, None, None) == L.EINVAL
    assert store(L.F32, 4, 4, P + 2, 4, P, P, None) == L.EALIGN      # below the element's alignment
    assert store(L.BF16, 4, 4, P, 4, P + 8, P, None) == L.EALIGN
    assert store(L.F32, (1 << 31) - 64, (1 << 31) - 64, P, 1 << 31, P, P, None) == L.ESHAPE
    assert store(L.F32, 0, 4, None, 4, None, None, None) == L.OK     # no rows: nothing enqueued
    assert lib.shampoo4_act8_load(L.F16, 4, 4, None, None, P, 4, None) == L.EINVAL
    assert lib.shampoo4_act8_load(L.F16, 4, 4, P, P, P, 2, None) == L.ESHAPE
    assert lib.shampoo4_act8_load(L.F16, 0, 4, None, None, None, 4, None) == L.OK


def test_activation_refusals():
    fwd, bwd = _lib().shampoo4_activation_forward, _lib().shampoo4_activation_backward
    n6 = [None] * 6
    assert fwd(2, L.F32, 4, 4, P, 4, None, 0, P, 4, *n6, None) == L.EINVAL
    assert fwd(0, 9, 4, 4, P, 4, None, 0, P, 4, *n6, None) == L.EINVAL
    assert fwd(0, L.F32, 4, 4, P, 2, None, 0, P, 4, *n6, None) == L.ESHAPE
    assert fwd(0, L.F32, 4, 4, P, 4, P, 3, P, 4, *n6, None) == L.ESHAPE
    assert fwd(0, L.F32, 4, 4, P, 4, None, 0, None, 4, *n6, None) == L.EINVAL
    assert fwd(0, L.F32, 4, 4, P, 4, None, 0, P, 4, P, None, None, None, None, None, None) == L.EINVAL
    assert fwd(0, L.F32, 4, 4, P, 4, None, 0, P, 4, None, None, P, P, None, None, None) == L.EINVAL   # up kept, no up
    assert fwd(0, L.F32, 4, 4, P, 4, None, 0, P, 4, P + 4, P, None, None, None, None, None) == L.EALIGN
    assert bwd(0, L.F32, 4, 4, P, 4, None, None, None, None, P, 4, None, 0, None) == L.EINVAL
    assert bwd(0, L.F32, 4, 4, P, 4, P, P, None, None, P, 4, P, 4, None) == L.EINVAL                  # dup, no up
    assert bwd(0, L.F32, 4, 4, P, 4, P, P, P, P, P, 4, None, 0, None) == L.EINVAL                     # up, no dup
    assert bwd(0, L.F32, 4, 4, P, 4, P, P, P, P, P, 4, P, 1, None) == L.ESHAPE
    assert bwd(0, L.F32, 0, 4, None, 4, None, None, None, None, None, 4, None, 0, None) == L.OK


def test_weight_grad_refusals():
    lib = _lib()
    f = lib.shampoo4_act8_weight_grad
    assert f(7, 4, 4, 4, 1.0, P, 4, P, P, 0.0, P, 4, None, 0, None) == L.EINVAL
    assert f(L.F32, 4, 0, 4, 1.0, P, 4, P, P, 0.0, P, 4, None, 0, None) == L.ESHAPE
    assert f(L.F32, 4, 4, 4, 1.0, P, 3, P, P, 0.0, P, 4, None, 0, None) == L.ESHAPE
    assert f(L.F32, 4, 4, 4, 1.0, P, 4, P, P, 0.0, P, 3, None, 0, None) == L.ESHAPE
    assert f(L.F32, 4, 4, 4, float("nan"), P, 4, P, P, 0.0, P, 4, None, 0, None) == L.EINVAL
    assert f(L.F32, 4, 4, 4, 1.0, P, 4, P, P, float("inf"), P, 4, None, 0, None) == L.EINVAL
    assert f(L.F32, 4, 4, 4, 1.0, P, 4, None, None, 0.0, P, 4, None, 0, None) == L.EINVAL
    assert f(L.F32, 4, 4, 4, 1.0, P, 4, P, P, 0.0, None, 4, None, 0, None) == L.EINVAL
    need = lib.shampoo4_act8_weight_grad_workspace_bytes(16384, 128, 128)      # few tiles, many rows: split
    assert need >= 2 * 128 * 128 * 4
    assert f(L.BF16, 16384, 128, 128, 1.0, P, 128, P, P, 0.0, P, 128, None, 0, None) == L.EINVAL
    assert f(L.BF16, 16384, 128, 128, 1.0, P, 128, P, P, 0.0, P, 128, P, need - 1, None) == L.ESMALLBUF
    assert f(L.BF16, 16384, 128, 128, 1.0, P, 128, P, P, 0.0, P, 128, P + 16, need, None) == L.EALIGN
    assert lib.shampoo4_act8_weight_grad_workspace_bytes(4, 0, 4) == 0
    # an output of many tiles fills the GPU without splitting its rows
    assert lib.shampoo4_act8_weight_grad_workspace_bytes(16384, 8192, 8192) == 0


def test_embedding_refusals():
    lib = _lib()
    f, g = lib.shampoo4_embedding, lib.shampoo4_embedding_grad
    assert f(L.F32, 2, 4, 9, 4, P, 4, P, 1.0, P, 4, None) == L.EINVAL          # id width
    assert f(L.F32, 8, 4, 0, 4, P, 4, P, 1.0, P, 4, None) == L.ESHAPE
    assert f(L.F32, 8, 4, 9, 4, P, 3, P, 1.0, P, 4, None) == L.ESHAPE
    assert f(L.F32, 8, 4, 9, 4, None, 4, P, 1.0, P, 4, None) == L.EINVAL
    assert f(L.F32, 8, 4, 9, 4, P, 4, None, 1.0, P, 4, None) == L.EINVAL
    assert f(L.F32, 8, 4, 9, 4, P, 4, P + 4, 1.0, P, 4, None) == L.EALIGN
    assert f(L.F32, 8, 0, 9, 4, P, 4, None, 1.0, None, 4, None) == L.OK
    need = lib.shampoo4_embedding_grad_workspace_bytes(100, 9, 4)
    assert need > 0 and need % 256 == 0
    assert g(L.F32, 8, 100, 9, 4, P, 4, P, 1.0, 0, P, 4, P, need - 1, None) == L.ESMALLBUF
    assert g(L.F32, 8, 100, 9, 4, P, 4, P, 1.0, 0, P, 4, None, 0, None) == L.EINVAL
    assert g(L.F32, 8, 100, 9, 4, P, 4, P, 1.0, 0, P, 2, P, need, None) == L.ESHAPE
    assert g(L.F32, 8, 100, 9, 4, P, 4, P, 1.0, 0, None, 4, P, need, None) == L.EINVAL
    assert g(L.F32, 8, 1 << 31, 9, 4, P, 4, P, 1.0, 0, P, 4, P, need, None) == L.ESHAPE
    # nothing to add: nothing is enqueued
    assert g(L.F32, 8, 0, 9, 4, None, 4, None, 1.0, 1, P, 4, None, 0, None) == L.OK


def test_policy_refusals():
    lib = _lib()
    f = lib.shampoo4_policy_loss
    need = lib.shampoo4_policy_loss_workspace_bytes(L.F32, 4, 9)
    assert need > 0

    def call(cfg=(0.2, 0.2, 0.0, 1.0), dtype=L.F32, idb=8, rows=4, vocab=9, z=P, ld=9, y=P, old=P, ref=None, adv=P,
             w=P, loss=P, logp=P, dz=P, ldd=9, ws=P, wsb=need):
        c = L.PolicyConfig(*cfg)
        return f(ctypes.byref(c), dtype, idb, rows, vocab, z, ld, y, old, ref, adv, w, loss, logp, dz, ldd, ws, wsb, None)

    for bad in ((-0.1, 0.2, 0.0, 1.0), (1.1, 0.2, 0.0, 1.0), (0.2, -1.0, 0.0, 1.0), (0.2, 0.2, -1.0, 1.0),
                (0.2, 0.2, 0.0, float("inf")), (float("nan"), 0.2, 0.0, 1.0), (0.2, float("inf"), 0.0, 1.0)):
        assert call(cfg=bad) == L.EINVAL, bad
    assert call(cfg=(0.2, 0.2, 0.1, 1.0)) == L.EINVAL           # KL without reference
    for k in ("z", "y", "old", "adv", "w", "loss"):
        assert call(**{k: None}) == L.EINVAL, k
    assert call(dtype=5) == L.EINVAL and call(idb=3) == L.EINVAL
    assert call(ld=8) == L.ESHAPE and call(ldd=8) == L.ESHAPE and call(vocab=0) == L.ESHAPE
    assert call(rows=1 << 23) == L.ESHAPE
    assert call(wsb=need - 1) == L.ESMALLBUF and call(ws=P + 8) == L.EALIGN and call(y=P + 4) == L.EALIGN
    assert lib.shampoo4_token_logprobs(L.F32, 8, 4, 9, P, 9, P, None, P, need, None) == L.EINVAL
    assert lib.shampoo4_token_logprobs(L.F32, 8, 0, 9, None, 9, None, None, None, 0, None) == L.OK


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    for f in (lambda: T.act8_store(x), lambda: T.activation_forward(x), lambda: T.embedding(x, torch.zeros(2, dtype=torch.int64)),
              lambda: T.token_logprobs(x, torch.zeros(4, dtype=torch.int64)), lambda: T.act8_load(None),
              lambda: T.act8_load(T.Act8.empty(4, 8, "cpu")), lambda: T.embedding_grad(x, torch.zeros(4), 3)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError):
        T.activation_forward(x, kind="relu")
    assert T.Act8.padded(33, 17) == (64, 32) and T.Act8.padded(0, 1) == (0, 16)


def test_oracle_checkpoint_properties():
    """The restored value is within half a step, the largest value keeps 7 bits, and values of
    the grid are fixed points."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((70, 5)) * 10.0 ** rng.uniform(-30, 30, (1, 5))
    x[:, 4] = 0
    codes, scales = o.act8_store(x)
    y = o.act8_load(codes, scales, 70, 5)
    step = np.repeat(2.0 ** (scales.astype(float) - 127), 32, 0)[:70, :5]
    assert np.all(np.abs(y - x) <= step / 2)
    for b in range(3):
        top = np.abs(codes[32 * b:32 * b + 32, :4]).max(0)
        assert np.all((top >= 63) & (top <= 127))
    c2, s2 = o.act8_store(y)
    assert np.array_equal(o.act8_load(c2, s2, 70, 5), y)
    assert np.all(codes[70:] == 0) and np.all(codes[:, 5:] == 0) and np.all(scales[:, 5:] == 1)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_oracle_activation_derivative_is_the_difference(kind):
    x = np.linspace(-8, 8, 401)
    h = 1e-5
    diff = (o.activation(x + h, kind) - o.activation(x - h, kind)) / (2 * h)
    assert np.max(np.abs(diff - o.activation_derivative(x, kind))) < 1e-9


def test_oracle_policy_gradient_is_the_difference():
    rng = np.random.default_rng(1)
    rows, vocab = 7, 11
    z = rng.standard_normal((rows, vocab))
    y = rng.integers(0, vocab, rows)
    lp = o.log_softmax(z)[np.arange(rows), y]
    # ratios on both sides of and inside the clip range, none at its ends
    old = lp - np.log(np.array([0.5, 0.9, 1.0, 1.1, 1.5, 0.7, 1.4]))
    adv = np.array([1.0, -1.0, 0.5, 2.0, 1.0, -1.0, -0.5])
    ref = lp + 0.3 * rng.standard_normal(rows)
    w = np.array([0.1, 0.2, 0.0, 0.1, 0.3, 0.1, 0.2])
    args = (y, old, adv, w, ref, 0.2, 0.28, 0.05)
    _, _, dz, _ = o.policy(z, *args)
    h = 1e-6
    for t in range(rows):
        for v in range(vocab):
            zp, zm = z.copy(), z.copy()
            zp[t, v] += h
            zm[t, v] -= h
            diff = (o.policy(zp, *args)[0] - o.policy(zm, *args)[0]) / (2 * h)
            assert abs(diff - dz[t, v]) < 1e-8
    assert np.all(dz[2] == 0)


def test_weight_grad_takes_every_output_that_a_launch_covers():
    """Up to 2^23 output tiles of 128 x 128 pass the check of shapes (and are refused here for their null operand)."""
    f = _lib().shampoo4_act8_weight_grad
    big = 1 << 18                                    # 2^22 tiles of 128 x 128, 2^24 of 64 x 64
    assert f(L.BF16, 4, big, big, 1.0, None, big, P, P, 0.0, P, big, None, 0, None) == L.EINVAL
    over = big // 2 * 3                              # above 2^23
    assert f(L.BF16, 4, over, over, 1.0, None, over, P, P, 0.0, P, over, None, 0, None) == L.ESHAPE
