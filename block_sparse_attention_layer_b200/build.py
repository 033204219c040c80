"""Build libvmoba.so (sm_100a) in-tree with nvcc.

Usage: python -m block_sparse_attention_layer_b200.build [--force] [-j N]

Every .cu file under csrc/ is compiled for sm_100a only
(-gencode arch=compute_100a,code=sm_100a) with -lineinfo and linked into
block_sparse_attention_layer_b200/libvmoba.so against the static CUDA
runtime; csrc/calls.cpp, the Python calls of norm_rope.py, is then compiled
against torch's headers into _calls.torch-<version>....so beside it, one for
each torch and Python (where that cannot be done a warning says why, and only
norm_rope's calls are missing).  Rebuilds only when a source or header is newer
than what was built from it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libvmoba.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libvmoba")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def calls_path() -> str:
    """The native Python calls (csrc/calls.cpp) of this interpreter and torch,
    both of which fix their binary interface."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_calls.torch-{torch.__version__}-{int(torch.compiled_with_cxx11_abi())}"
                             f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_calls(force: bool = False) -> str:
    """Compile csrc/calls.cpp against the installed torch."""
    calls = calls_path()
    src = os.path.join(CSRC, "calls.cpp")
    deps = [src, *glob.glob(os.path.join(ROOT, "include", "*.h"))]
    if not force and os.path.exists(calls) and \
            all(os.path.getmtime(p) <= os.path.getmtime(calls) for p in deps):
        return calls
    if os.path.exists(calls):
        os.remove(calls)                # of an older source: must not be taken for this one's
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    include = [sysconfig.get_path("include"), os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", *("-I" + i for i in include),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", src,
           "-o", calls + ".tmp", "-L" + os.path.join(root, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for {src}:\n{r.stderr}")
    os.replace(calls + ".tmp", calls)
    return calls


def build(force: bool = False, jobs: int = 0, verbose_ptxas: bool = False) -> str:
    path = build_library(force, jobs, verbose_ptxas)
    try:
        build_calls(force)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the Python calls of norm_rope are not built: {e}", RuntimeWarning)
    return path


def build_library(force: bool = False, jobs: int = 0, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=0)
    ap.add_argument("--ptxas-v", action="store_true", help="print register/smem usage")
    a = ap.parse_args()
    print(build(force=a.force, jobs=a.j, verbose_ptxas=a.ptxas_v))


if __name__ == "__main__":
    main()
