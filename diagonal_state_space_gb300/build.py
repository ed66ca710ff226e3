"""Builds libs5.so in-tree with nvcc for sm_103a (one -gencode, no cmake), and
the binding's native half with g++ against the installed torch (where there is
one: the library needs nvcc alone).

Translation units compile in parallel into ``_build/`` at the repository root
and link into ``diagonal_state_space_gb300/libs5.so`` and ``_marshal.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libs5.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]

LINK_LIBS: list[str] = []


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libs5.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, what):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, res.stdout, res.stderr))


def _has_torch() -> bool:
    """Whether there is a torch with CUDA to build the binding for; the library itself is for C callers too."""
    try:
        import torch
    except ImportError:
        return False
    return torch.version.cuda is not None


def _binary_interface() -> str:
    """What the binding's compiled half depends on: torch, Python and the C++ library's interface."""
    import torch
    return "%s-%s-abi%d" % (torch.__version__, sysconfig.get_config_var("SOABI"), torch._C._GLIBCXX_USE_CXX11_ABI)


def _marshal_object(force: bool) -> str:
    """csrc/marshal.cpp for the torch and the Python that are installed (part of the object's name)."""
    import torch
    src = os.path.join(CSRC, "marshal.cpp")
    obj = os.path.join(OBJ, "marshal-%s.o" % _binary_interface())
    if force or _stale(obj, [src, os.path.join(ROOT, "include", "s5.h")]):
        cuda = os.path.dirname(os.path.dirname(_nvcc()))
        _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
              "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", os.path.join(ROOT, "include"),
              "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(torch.__file__), "include"),
              "-I", os.path.join(cuda, "include"), "-c", src, "-o", obj], "g++ for %s" % src)
    return obj


def _linked_from(obj: str) -> bool:
    """Whether _marshal.so comes from this object: a later object of another torch says nothing about it."""
    try:
        with open(os.path.join(OBJ, "marshal.linked")) as f:
            return f.read() == os.path.basename(obj) and not _stale(MARSHAL, [obj])
    except OSError:
        return False


def _link_marshal(obj: str) -> None:
    import torch
    tmp = MARSHAL + ".tmp%d" % os.getpid()
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", PKG, "-ls5", "-Wl,-rpath,$ORIGIN"], "link of _marshal.so")
    os.replace(tmp, MARSHAL)
    with open(os.path.join(OBJ, "marshal.linked"), "w") as f:
        f.write(os.path.basename(obj))


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(OBJ, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    srcs = sources()
    objs = [os.path.join(OBJ, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        if not force and not _stale(obj, [src, *headers]):
            return obj
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, res.stdout, res.stderr))
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        marshal = ex.submit(_marshal_object, force) if _has_torch() else None
        list(ex.map(compile_one, zip(srcs, objs)))
        _link_library(nvcc, objs, force)     # needs nothing of torch: it is there whatever becomes of the binding
        marshal = marshal and marshal.result()
    if marshal and (force or not _linked_from(marshal)):
        _link_marshal(marshal)
    return LIB


def _link_library(nvcc: str, objs: list[str], force: bool) -> None:
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-cudart", "static",
               "-o", tmp, *objs, *LINK_LIBS]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (res.stdout, res.stderr))
        os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
