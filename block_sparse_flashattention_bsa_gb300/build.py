"""Build libbsa.so (the CUDA kernels + C ABI) in-tree with nvcc for sm_103a,
and _bsa_torch.so (compiled marshalling of the projection and paged-cache
calls, linked against it) with the host compiler.

Usage: ``python -m block_sparse_flashattention_bsa_gb300.build [--force]``.
Translation units compile in parallel into ``_build/`` at the repository
root; the shared library lands next to this file.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbsa.so")
BINDING = os.path.join(PKG, "_bsa_torch.so")
BINDING_SOURCE = "bsa_torch.cpp"
BINDING_RECORD = "bsa_torch.made_for"  # in BUILD: the torch and the Python that the binding was compiled for

SOURCES = ["bsa_api.cu", "bsa_fwd.cu", "bsa_mask.cu", "bsa_topk.cu", "bsa_noalloc.cu", "bsa_pair.cu", "bsa_bwd.cu", "bsa_fp8.cu", "bsa_shard.cu",
           "bsa_rope.cu", "bsa_cache.cu", "bsa_tree.cu"]
HEADERS = ["bsa_ptx.cuh", "bsa_internal.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _fresh(target: str, sources) -> bool:
    """Whether target is there and no older than its sources."""
    paths = [os.path.join(CSRC, s) for s in sources] + [os.path.join(INCLUDE, "bsa.h")]
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(p) for p in paths)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _compile_binding() -> str:
    import sysconfig

    torch = _torch()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    troot = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "bsa_torch.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", os.path.join(troot, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(cuda, "include"), "-I", INCLUDE, "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (BINDING_SOURCE, r.stdout, r.stderr))
    return obj


def _link(cmd, out: str) -> None:
    tmp = out + ".tmp.%d" % os.getpid()
    r = subprocess.run([x if x != out else tmp for x in cmd], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, out)


def _torch():
    try:
        import torch
        return torch
    except ImportError:
        return None


def _made_for() -> str:
    torch = _torch()
    return "%s\n%s\n%s\n" % (torch.__version__, os.path.dirname(torch.__file__), sys.version)


def _binding_fresh() -> bool:
    try:
        with open(os.path.join(BUILD, BINDING_RECORD)) as f:
            return f.read() == _made_for() and _fresh(BINDING, [BINDING_SOURCE])
    except OSError:
        return False


def _link_binding(obj: str) -> None:
    tlib = os.path.join(os.path.dirname(_torch().__file__), "lib")
    _link([os.environ.get("CXX", "g++"), "-shared", "-o", BINDING, obj, "-L" + tlib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + PKG, "-l:libbsa.so", "-Wl,-rpath,$ORIGIN",
           "-Wl,-rpath," + tlib], BINDING)
    with open(os.path.join(BUILD, BINDING_RECORD), "w") as f:
        f.write(_made_for())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Builds what is missing or older than its sources (the binding also where
    torch or Python is not what it was compiled for).  libbsa.so needs nvcc
    alone and is linked whether or not _bsa_torch.so can be; without torch,
    which _bsa_torch.so is for, only libbsa.so is built."""
    lib = force or not _fresh(LIB, SOURCES + HEADERS)
    binding = _torch() is not None and (force or not _binding_fresh())
    if not lib and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bobj = ex.submit(_compile_binding) if binding else None
        if lib:
            objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
            _link([nvcc(), *ARCH, "-shared", "-o", LIB, *objs, "-lcudart_static", "-lrt", "-lpthread", "-ldl"], LIB)
        if binding:
            _link_binding(bobj.result())
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register / spill / smem use")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.ptxas_v))
