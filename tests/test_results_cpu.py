"""Two results of a call in the same memory are refused, before anything reaches a device."""

import ctypes
import os

import pytest

from bit_quantized_shampoo_amd import _lib as L

A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000      # aligned addresses that no refused call may touch


def _lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return L.lib()


def _config():
    return ctypes.byref(L.BlockNormConfig(1e-6, 1.0, L.DropoutConfig(0.0, 0, 0, 0, None)))


def test_a_weight_over_its_transpose():
    f = _lib().shampoo4_fp8_store_weight
    assert f(L.F32, 4, 4, A, 4, B, C, B, D, None) == L.EINVAL
    assert f(L.F32, 4, 4, A, 4, B, C, D, C, None) == L.EINVAL
    assert f(L.F32, 0, 4, None, 4, B, C, B, C, None) == L.OK


def test_the_norm_over_the_sum():
    f = _lib().shampoo4_block_norm_forward
    for x, h, out, y in ((A, B, C, C), (A, B, A, A), (A, B, B, B)):
        assert f(_config(), L.F32, 4, 8, x, 8, h, 8, None, None, 0, 0, D, out, 8, y, 8, None, None, None, None, None) == L.EINVAL


def test_one_gradient_over_another():
    lib = _lib()
    need = lib.shampoo4_block_norm_workspace_bytes(4, 8)
    for rows, dx, dh, dgate in ((4, C, C, None), (4, C, D, C), (4, C, D, D), (4, B, B, None)):
        assert lib.shampoo4_block_norm_backward(_config(), L.F32, rows, 8, A, 8, B, 8, A, 8, D, D, A, 8, None, None, A, 1, 8, dx, 8,
                                                dh, 8, D, None, dgate, 8, A, need, None) == L.EINVAL
