"""Build libsfa.so in-tree with nvcc for sm_100a (B200), and the extension module _bind.so.

    python -m frame_sparse_attention_b200.build [--force] [--verbose-ptxas]

Each csrc/*.cu is compiled to an object under _build/ (rebuilt when it or a header
changed), then linked into frame_sparse_attention_b200/libsfa.so with the CUDA
runtime linked statically; csrc/sfa_bind.cpp, the binding of the 8-bit frame cache's calls,
is built with the C++ compiler against PyTorch's headers and libsfa.so (again when PyTorch or
the interpreter changed: _build/sfa_bind.built_for says what it was built for).  No GPU is
needed to build.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsfa.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_SRC = os.path.join(CSRC, "sfa_bind.cpp")
BIND_BUILT_FOR = os.path.join(OBJDIR, "sfa_bind.built_for")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsfa.so")


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    hdrs += glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def _bind_target() -> str:
    """What _bind.so's object layout depends on beside its source: PyTorch, its C++ ABI, the interpreter."""
    import torch
    return (f"torch {torch.__version__} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"python {sysconfig.get_config_var('SOABI')}")


def _bind_fresh(target: str) -> bool:
    if not (os.path.exists(BIND) and os.path.exists(BIND_BUILT_FOR)):
        return False
    with open(BIND_BUILT_FOR) as f:
        built_for = f.read()
    return built_for == target and os.path.getmtime(BIND) >= max(os.path.getmtime(BIND_SRC), _newest_header())


def _build_bind(nvcc: str, force: bool) -> None:
    """_bind.so, with torch's own libraries as they are loaded already by `import torch`."""
    target = _bind_target()
    if not force and _bind_fresh(target):
        return
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    inc = [INCLUDE, *include_paths(), cuda, sysconfig.get_paths()["include"]]
    tmp = BIND + f".tmp{os.getpid()}"
    subprocess.check_call([shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-shared",
                           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                           *(f"-isystem{i}" for i in inc), BIND_SRC, "-o", tmp,
                           *(f"-L{i}" for i in library_paths()), f"-L{PKG}", "-l:libsfa.so", "-Wl,-rpath,$ORIGIN",
                           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    os.replace(tmp, BIND)
    with open(BIND_BUILT_FOR, "w") as f:
        f.write(target)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    flags = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        stale = (force or verbose_ptxas or not os.path.exists(obj)
                 or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time))
        if stale:
            subprocess.check_call([nvcc, *flags, "-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    _build_bind(nvcc, force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose_ptxas=args.verbose_ptxas))
