"""Kernels that need more than 64 KB of LDS on every device of a process, without a GPU: the library runs against a
stand-in for the runtime's launch calls, which holds what the runtime holds, a kernel's limit of dynamic LDS for the
device that was current when it was raised."""

import os
import subprocess
import sys

import pytest

from bit_quantized_shampoo_amd import _lib as L

RUNTIME = r"""
#include <cstddef>
#include <map>
#include <utility>
extern "C" {
struct dim3 { unsigned x, y, z; };
static std::map<std::pair<const void*, int>, size_t> limits;
static int device = 0, failures = 0, launches = 0, large = 0, refused = 0, last = 0;
static dim3 grid, block;
static size_t lds;
static void* queue;
void stand_in(int dev, int fail) { device = dev; failures = fail; }
int stand_in_launches() { return launches; }
int stand_in_large() { return large; }
int stand_in_refused() { return refused; }
int hipGetDevice(int* d) { *d = device; return 0; }
int hipGetLastError() { int e = last; last = 0; return e; }
int hipFuncSetAttribute(const void* f, int, int value) {
    if (failures > 0) { --failures; return 2; }
    limits[{f, device}] = value;
    return 0;
}
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, void* q) { grid = g; block = b; lds = s; queue = q; return 0; }
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* s, void** q) { *g = grid; *b = block; *s = lds; *q = queue; return 0; }
int hipLaunchKernel(const void* f, dim3, dim3, void**, size_t s, void*) {
    ++launches;
    large += s > 65536;
    if (s > 65536 && limits[{f, device}] < s) { ++refused; return last = 1; }
    return 0;
}
}
"""

CALLS = r"""
import ctypes, sys
rt = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
P, Q, I, F = ctypes.c_void_p(0x10000), ctypes.c_int64, ctypes.c_int, ctypes.c_float
lib.shampoo4_act8_weight_grad_workspace_bytes.restype = ctypes.c_size_t
BF16, OK, EHIP = (int(a) for a in sys.argv[3:])

def product(t, n, k):
    return lib.shampoo4_fp8_linear(I(BF16), I(BF16), Q(t), Q(n), Q(k), None, Q(0), P, P, P, P, I(0), P, Q(n), None,
                                   ctypes.c_size_t(0), None)

def weight_grad(t, n, c):
    need = lib.shampoo4_act8_weight_grad_workspace_bytes(Q(t), Q(n), Q(c))
    return lib.shampoo4_act8_weight_grad(I(BF16), Q(t), Q(n), Q(c), F(1), P, Q(n), P, P, F(0), P, Q(c), P,
                                         ctypes.c_size_t(need), None)

calls = [lambda: product(4096, 4096, 1152), lambda: product(2048, 2048, 256), lambda: weight_grad(16384, 4096, 4096),
         lambda: weight_grad(200, 300, 300)]
for dev in (0, 1, 0, 7):
    rt.stand_in(dev, 0)
    got = [f() for f in calls]
    assert got == [OK] * 4, (dev, got)
assert rt.stand_in_large() >= 12 and rt.stand_in_refused() == 0
n = rt.stand_in_launches()
rt.stand_in(3, 1)                       # a limit that cannot be raised is an error, and is raised by the next call
assert product(4096, 4096, 1152) == EHIP and rt.stand_in_launches() == n
assert product(4096, 4096, 1152) == OK and rt.stand_in_launches() == n + 1
print("done")
"""


def test_limits_of_lds_belong_to_a_device(tmp_path):
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    src, so, calls = tmp_path / "runtime.cpp", tmp_path / "runtime.so", tmp_path / "calls.py"
    src.write_text(RUNTIME)
    calls.write_text(CALLS)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", so, src], check=True)
    run = subprocess.run([sys.executable, calls, so, L.LIB_PATH, str(L.BF16), str(L.OK), str(L.EHIP)], capture_output=True,
                         text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "done", run.stderr
