"""Build libvimscan.so (HIP, gfx950) in-tree with hipcc, and _binding.so, the
torch side of some of its entry points, with the host compiler."""
from __future__ import annotations

import os
import re
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "vimscan.hip")
SRCS = [SRC] + [os.path.join(PKG, "csrc", f) for f in
                ("proj.hip", "causal.hip", "causal_grad.hip", "beam.hip", "gated.hip",
                 "norm.hip", "vocab.hip", "host.cpp", "host_causal.cpp", "host_model.cpp")]
LIB = os.path.join(PKG, "libvimscan.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING_SRC = os.path.join(PKG, "csrc", "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    # packed-fp32 VALU forms are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else "hipcc"


def scratch_kernels(log: str):
    """Kernels whose resource-usage remark reports scratch memory: register
    arrays that did not stay in registers (a step left out of line, a
    dynamic index), which costs an order of magnitude in time."""
    bad, name = [], None
    for line in log.splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            continue
        m = re.search(r"ScratchSize \[bytes/lane\]: (\d+)", line)
        if m and int(m.group(1)) > 0:
            bad.append((name, int(m.group(1))))
    return bad


def build(out: str = LIB, extra=()) -> str:
    """Compile every source for itself, at most one compiler per CPU at a
    time, and link the objects."""
    tmp = out + ".tmp%d" % os.getpid()
    flags = [*HIPCC_FLAGS, "-Rpass-analysis=kernel-resource-usage", *extra, "-I", INCLUDE]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, "%d.o" % i) for i in range(len(SRCS))]

        def compile_one(i):
            return subprocess.run([hipcc(), *flags, "-c", SRCS[i], "-o", objs[i]],
                                  capture_output=True, text=True)

        with ThreadPoolExecutor(min(len(SRCS), os.cpu_count() or 1)) as pool:
            done = list(pool.map(compile_one, range(len(SRCS))))
        for src, r in zip(SRCS, done):
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError("hipcc failed compiling %s" % src)
        bad = scratch_kernels("\n".join(r.stderr for r in done))
        if bad:
            raise RuntimeError("kernels use scratch memory: " +
                               ", ".join("%s (%d B/lane)" % b for b in bad))
        r = subprocess.run([hipcc(), "-shared", "--offload-arch=gfx950", *objs, "-o", tmp],
                           capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("hipcc failed linking %s" % out)
    os.replace(tmp, out)
    return out


def build_binding(out: str = BINDING) -> str:
    """Compile _binding.so against the installed torch."""
    import torch

    home = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    tmp = out + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-unused-function",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", INCLUDE, "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(rocm, "include"), "-isystem", sysconfig.get_paths()["include"],
           BINDING_SRC, "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("the host compiler failed on %s" % BINDING_SRC)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build())
    print(build_binding())
