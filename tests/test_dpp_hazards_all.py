"""The DPP read rule (tests/test_dpp_hazards.py) on every code object of the
library: each HIP source is compiled for itself, so the library's fat binary
holds one bundle per source, and that test reads the first."""
import os
import subprocess
import tempfile

import pytest

import test_dpp_hazards as rule

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "vision_mamba_selective_amd", "libvimscan.so")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def bundles():
    with tempfile.TemporaryDirectory() as d:
        fat = os.path.join(d, "fatbin")
        subprocess.run([os.path.join(rule.LLVM, "llvm-objcopy"), "--dump-section", ".hip_fatbin=" + fat, LIB,
                        os.path.join(d, "copy.so")], check=True, capture_output=True)
        data = open(fat, "rb").read()
    at = []
    i = data.find(MAGIC)
    while i >= 0:
        at.append(i)
        i = data.find(MAGIC, i + 1)
    return [data[a:b] for a, b in zip(at, at[1:] + [len(data)])]


def functions(bundle):
    """rule.disassemble for one bundle: it reads a library's .hip_fatbin section, so the bundle is put into one."""
    with tempfile.TemporaryDirectory() as d:
        part, src, lib = (os.path.join(d, n) for n in ("part", "e.c", "e.so"))
        with open(part, "wb") as f:
            f.write(bundle)
        open(src, "w").close()
        subprocess.run(["gcc", "-shared", "-o", lib, src], check=True, capture_output=True)
        out = os.path.join(d, "with.so")
        subprocess.run([os.path.join(rule.LLVM, "llvm-objcopy"), "--add-section", ".hip_fatbin=" + part, lib, out],
                       check=True, capture_output=True)
        return rule.disassemble(out)


@pytest.mark.skipif(not os.path.exists(LIB), reason="the library is not built")
def test_every_code_object_honours_the_dpp_rule():
    found = bundles()
    assert len(found) >= 5
    names = []
    for b in found:
        funcs = functions(b)
        names += funcs
        result = rule.violations(funcs)
        bad = result[0] if isinstance(result, tuple) else result
        assert not bad, bad[:5]
    for kernel in ("rowscan_kernel", "causal_scan_kernel", "causal_scan4_kernel", "causal_grad_kernel",
                   "adjoint_carry_kernel", "beam_part_kernel"):
        assert any(kernel in n for n in names), kernel
