"""Build libdq.so in-tree with hipcc for gfx950, and _bind.so, the compiled part of its Python
binding.

    python -m dual_scale_w4a4_amd.build

The library needs hipcc alone. The binding is built against torch's headers; where torch is not
installed there is nothing for it to bind to, and it is left out.

Flags: IEEE fp32 arithmetic exactly as written (-ffp-contract=off: no fused multiply-add
unless the source asks for one; subnormals kept), and packed-fp32 instruction selection
disabled.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB_PATH = os.path.join(HERE, "libdq.so")
BIND_PATH = os.path.join(HERE, "_bind.so")
SOURCES = ["dq_kernels.hip", "dq_pass.hip", "dq_rowres.hip", "dq_act.hip", "dq_gemm.hip",
           "dq_norm.hip", "dq_mlp.hip",
           "dq_api.hip"]
ARCH = os.environ.get("DQ_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Werror=return-type",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "hipcc"


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building libdq.so or _bind.so")


def cxx() -> str:
    """The host compiler: CXX, g++, or else the clang++ that hipcc itself runs."""
    cand = os.environ.get("CXX") or shutil.which("g++")
    rocm = os.path.dirname(os.path.dirname(shutil.which(hipcc()) or hipcc()))
    return cand or os.path.join(rocm, "llvm", "bin", "clang++")


def bind_cmd(out: str):
    """The compiler call for the Python binding of the MLP operators (host code only, against
    torch's headers and the libdq.so beside it)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [f"-I{p}" for p in (*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
                              os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include"))]
    return [cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            "-D__HIP_PLATFORM_AMD__",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc,
            os.path.join(CSRC, "dq_bind.cpp"), "-o", out, f"-L{tlib}", "-ltorch_python",
            "-ltorch_cpu", "-lc10", f"-L{HERE}", "-l:libdq.so", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False) -> str:
    """Compile every source to an object in parallel (no device code crosses files), then
    link the shared library and build the Python binding that calls it, if there is a torch."""
    from concurrent.futures import ThreadPoolExecutor

    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    objs = [os.path.join(objdir, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    cmds = [[hipcc(), *compile_flags, "-c", os.path.join(CSRC, s), "-o", o]
            for s, o in zip(SOURCES, objs)]
    workers = max(1, min(len(cmds), int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))
    with ThreadPoolExecutor(max_workers=workers) as ex:
        for f in [ex.submit(_run, c, verbose) for c in cmds]:
            f.result()
    _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", LIB_PATH + ".tmp"],
         verbose)
    os.replace(LIB_PATH + ".tmp", LIB_PATH)
    try:
        import torch  # noqa: F401
    except ImportError:
        print("torch is not installed: libdq.so without its Python binding", file=sys.stderr)
        if os.path.exists(BIND_PATH):  # of an older library
            os.remove(BIND_PATH)
        return LIB_PATH
    _run(bind_cmd(BIND_PATH + ".tmp"), verbose)
    os.replace(BIND_PATH + ".tmp", BIND_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
