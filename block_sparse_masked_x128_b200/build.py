"""Build the sm_100a shared library in-tree: block_sparse_masked_x128_b200/_lib/libfa_b200.so.

    python block_sparse_masked_x128_b200/build.py [--verbose] [--ptxas-info] [--force] [--debug]

(Run it as a file, not as a package module: importing the package loads the library.)

Beside it goes _lib/fa_b200_torch.so, the host path of the Python serving calls (g++ against torch's
headers; left out where torch is not installed: the library does not need it).
Each .cu file is compiled to an object in parallel (nvcc cross-compiles for sm_100a without
a GPU), then linked into one shared library exporting the C ABI of include/fa_b200.h.
Objects are rebuilt only when a source or header is newer.  `--ptxas-info` prints the
registers and shared memory of every kernel (nvcc -Xptxas -v).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libfa_b200.so")
TRACE_LIB = os.path.join(LIBDIR, "libfa_b200_trace.so")
DEBUG_LIB = os.path.join(LIBDIR, "libfa_b200_debug.so")
BINDING = os.path.join(LIBDIR, "fa_b200_torch.so")      # the serving calls' host path (csrc/binding.cpp)
SOURCES = ["api.cu", "mask_builder.cu", "attn_fwd.cu", "noalloc.cu", "masked_softmax.cu", "attn_bwd.cu", "decode.cu",
           "serving_api.cu", "rotary.cu", "kv_cache.cu", "decode_cache.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(ptxas_info: bool, trace: bool = False, debug: bool = False) -> list:
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if ptxas_info:
        f += ["-Xptxas", "-v"]
    if trace:
        f += ["-DFA_TRACE"]
    if debug:
        f += ["-DFA_DEBUG"]
    return f


def _headers() -> list:
    hs = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, h) for h in os.listdir(INCLUDE) if h.endswith(".h")]


def _compile(src: str, flags: list, force: bool, build_dir: str = BUILD) -> tuple:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    srcp = os.path.join(CSRC, src)
    newest = max(os.path.getmtime(p) for p in [srcp] + _headers())
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj, ""
    cmd = [_nvcc()] + flags + ["-c", srcp, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def build_binding(force: bool = False) -> Optional[str]:
    """Compile csrc/binding.cpp, the Python extension that takes torch tensors to the C ABI.  None where
    torch is not installed."""
    try:
        import torch
    except ModuleNotFoundError as e:
        if e.name != "torch":
            raise
        return None
    import sysconfig
    src = os.path.join(CSRC, "binding.cpp")
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"), src, "-o", BINDING,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    # Current: newer than its sources and made by this command (wherever the tree lies) against this
    # torch and Python.
    made = "\n".join([*cmd, torch.__version__, str(torch.version.git_version), sys.version]).replace(ROOT, "")
    stamp = os.path.join(BUILD, "fa_b200_torch.made")
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "fa_b200.h")))
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == made:
                return BINDING
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made)
    return BINDING


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False,
          trace: bool = False, debug: bool = False) -> str:
    """Build the library; trace=True builds the phase-tracing variant, debug=True the variant
    whose kernels check metadata indices (FA_DEBUG), each under its own name."""
    variant = "trace" if trace else ("debug" if debug else "")
    build_dir = os.path.join(BUILD, variant) if variant else BUILD
    lib = TRACE_LIB if trace else (DEBUG_LIB if debug else LIB)
    os.makedirs(build_dir, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    flags = _flags(ptxas_info, trace, debug)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(lambda s: _compile(s, flags, force or ptxas_info, build_dir), SOURCES))
    objs = [o for o, _ in results]
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                print(log)
    newest_obj = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(lib) or os.path.getmtime(lib) < newest_obj:
        cmd = [_nvcc()] + ARCH + ["-shared", "-o", lib] + objs + ["-lcudart_static", "-ldl", "-lrt", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    # Last, so that whatever the binding lacks, the library is there.
    if binding.result() is None and verbose:
        print("torch is not installed: fa_b200_torch.so (the Python serving calls) is left out")
    return lib


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--trace", action="store_true", help="build the phase-tracing variant")
    ap.add_argument("--debug", action="store_true",
                    help="build the variant whose kernels check metadata indices (FA_DEBUG)")
    a = ap.parse_args(argv)
    print(build(a.verbose, a.ptxas_info, a.force, a.trace, a.debug))
    return 0


if __name__ == "__main__":
    sys.exit(main())
