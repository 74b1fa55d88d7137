"""What the compiler does not check of inline assembly: the clobbers that a statement declares, from the sources, and
the states between its instructions and what the compiler put before them, from the listing of the built object."""

import glob
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "bit_quantized_shampoo_amd")
LLVM = "/opt/rocm/llvm/bin"


def _statements():
    """(file, text) of every asm statement."""
    for path in sorted(glob.glob(os.path.join(PKG, "csrc", "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\b\s*(volatile)?\s*\(", text):
            end, depth = m.end(), 1
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            yield os.path.basename(path), text[m.start():end]


def test_m0_is_declared():
    """A statement that writes m0 says so."""
    found = [(name, s) for name, s in _statements() if re.search(r"\bs_\w+ m0\b", s)]
    assert found
    for name, s in found:
        assert re.search(r':\s*"m0"\s*\)$', s), (name, s)


def _registers(text):
    """{(kind, number)} of the v, a and s registers that a piece of a listing names."""
    out = set()
    for kind, lo, hi, kind1, one in re.findall(r"\b([vas])\[(\d+):(\d+)\]|\b([vas])(\d+)\b", text):
        out |= {(kind, i) for i in range(int(lo), int(hi) + 1)} if kind else {(kind1, int(one))}
    return out


def _listing(tmp_path, source):
    obj = os.path.join(PKG, "_build", source.replace(".hip", ".o"))
    tools = [os.path.join(LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump")]
    if not os.path.exists(obj) or not all(map(os.path.exists, tools)):
        pytest.skip("the objects are not built here (run __graft_entry__.build())")
    fat, code = str(tmp_path / "fat"), str(tmp_path / "code")
    subprocess.run([tools[0], f"--dump-section=.hip_fatbin={fat}", obj, str(tmp_path / "rest")], check=True)
    subprocess.run([tools[1], "--unbundle", "--type=o", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={fat}",
                    f"--output={code}"], check=True)
    return subprocess.run([tools[2], "-d", "--no-show-raw-insn", code], check=True, capture_output=True, text=True).stdout


def test_states_before_assembly(tmp_path):
    """Of the kernels whose loads to LDS and matrix instructions are written as assembly: a load reads no scalar
    register that a vector instruction wrote less than five states before, and a matrix instruction no vector register
    that one wrote less than two states before.  (The compiler's own are among what is looked at.)"""
    loads = products = 0
    before = []                                   # (registers written by a vector instruction, states it takes)
    for line in _listing(tmp_path, "linear.hip").splitlines():
        if line.endswith(">:"):
            before = []
            continue
        t = line.split("//")[0].strip()
        if not re.match(r"[a-z]\w+", t) or ":" in t.split()[0]:
            continue
        op, _, rest = t.partition(" ")
        args = [a.strip() for a in re.split(r",(?![^\[]*\])", rest)]
        mfma = op.startswith("v_mfma")
        need, reads = 0, set()
        if op.startswith("buffer_load"):
            loads += 1
            need, reads = 5, {r for r in _registers(rest) if r[0] == "s"}
        elif mfma:
            products += 1
            need, reads = 2, _registers(",".join(args[1:]))
        states = 0
        for written, taken in reversed(before):
            if states >= need:
                break
            assert not written & reads, (states, line)
            states += taken
        taken = int(rest, 0) + 1 if op == "s_nop" else 1
        vector = op.startswith("v_") and not mfma
        before = (before + [(_registers(args[0]) if vector else set(), taken)])[-8:]
    assert loads > 50 and products > 500
