"""Build libtpfuse.so in-tree with hipcc for gfx950.

Usage: python -m tensor_gemm_reduction_amd.build   (or build() from Python)
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import time

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libtpfuse.so")
ARGS = os.path.join(LIBDIR, "_args.so")      # the Python binding's native argument checks

SOURCES = ["tpf_kernels.hip", "tpf_api.cpp", "tpf_block_api.cpp", "tpf_norm.hip", "tpf_stash.hip",
           "tpf_stash_grad.hip", "tpf_qweight.hip", "tpf_scaled_api.cpp", "tpf_scaled_pack.hip", "tpf_scaled_matmul.hip",
           "tpf_scaled_few.hip", "tpf_experts.hip"]
HEADERS = ["tpf_device.hpp", "tpf_internal.hpp", "tpf_gemm.hpp", "tpf_stationary.hpp", "tpf_host.hpp",
           "tpf_block.hpp", "tpf_tiles.hpp", "tpf_scaled.hpp", "tpf_scaled_device.hpp", "tpf_gauss.hpp"]

# Packed-fp32 instructions are disabled for all device code: the compiler
# would otherwise form v_pk_* fp32 ops from plain float code.
HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-result",
    "-I" + os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libtpfuse)")


# tpf_kernels.hip is compiled as KERNEL_PARTS translation units (-DTPF_PART=n),
# in parallel; see the part list at the top of that file.
KERNEL_PARTS = 9


def _compile_jobs(cc: str):
    jobs = []
    for part in range(KERNEL_PARTS):
        obj = os.path.join(LIBDIR, f"tpf_kernels_p{part}.o")
        jobs.append((f"tpf_kernels.hip (part {part})", obj,
                     [cc, "-x", "hip", "-c", os.path.join(CSRC, "tpf_kernels.hip"), "-o", obj,
                      f"-DTPF_PART={part}"] + HIPCC_FLAGS))
    for src in SOURCES:
        if src == "tpf_kernels.hip":
            continue
        obj = os.path.join(LIBDIR, os.path.splitext(src)[0] + ".o")
        jobs.append((src, obj, [cc, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + HIPCC_FLAGS))
    return jobs


def _args_command(out: str):
    """Compile command of the argument checks: host code against torch's headers."""
    import torch
    from torch.utils import cpp_extension
    include = cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]
    return (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             os.path.join(CSRC, "tpf_args.cpp"), "-o", out] + [f"-I{i}" for i in include]
            + ["-L" + cpp_extension.TORCH_LIB_PATH, "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10"])


def _start(name: str, cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    return name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)


def _failure(name: str, pr, verbose: bool):
    """What a finished compiler said if it failed, else None."""
    out, err = pr.communicate()
    if pr.returncode != 0:
        return f"compiling {name} failed:\n{out}\n{err}"
    if verbose and err.strip():
        print(err, file=sys.stderr)
    return None


def build(verbose: bool = False) -> str:
    """Compile every source for gfx950, link libtpfuse.so and the binding's
    argument checks; returns the library's path.  The checks need g++ and
    torch's headers: where they do not build, the library is there all the same
    when the error is raised."""
    os.makedirs(LIBDIR, exist_ok=True)
    cc = hipcc()
    t0 = time.time()
    jobs = _compile_jobs(cc)
    procs = [_start(name, cmd, verbose) for name, _, cmd in jobs]
    args_tmp, args_failed = ARGS + ".tmp", None
    try:
        args = _start("tpf_args.cpp", _args_command(args_tmp), verbose)
    except (ImportError, OSError) as e:      # no torch, no g++
        args, args_failed = None, f"{type(e).__name__}: {e}"
    failed = [f for f in (_failure(name, pr, verbose) for name, pr in procs) if f]
    if args is not None:
        args_failed = _failure(*args, verbose)
    if failed:
        raise RuntimeError("\n".join(failed))
    objs = [obj for _, obj, _ in jobs]
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-fPIC", "--offload-arch=gfx950", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    if args_failed:
        raise RuntimeError(f"{LIB} is built, but not {ARGS} (the MLP block's calls need it): {args_failed}")
    os.replace(args_tmp, ARGS)
    if verbose:
        print(f"built {LIB} in {time.time() - t0:.1f}s", flush=True)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
