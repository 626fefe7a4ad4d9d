"""Build libpgd.so in-tree for sm_103a.

Each CUDA translation unit is compiled by nvcc with one -gencode
(compute_103a -> sm_103a), in parallel, and the objects are linked into
``paged_gqa_decode_kv_gb300/_build/libpgd.so`` (CUDA runtime linked
statically); this needs the CUDA toolkit and a C++ compiler alone.  Beside it,
where torch is installed, ``_pgd_tensors``: the part of the binding that reads
torch tensors, a CPython extension built against that torch (whose version is
part of its file name).  Rebuilds only when a source or header is newer than
what is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpgd.so")
HEADER = os.path.join(ROOT, "include", "pgd.h")
TENSORS_SRC = os.path.join(HERE, "binding", "tensors.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-Wall",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _has_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def tensors_path() -> str:
    """The binding's tensor extension for the installed torch."""
    import torch

    tag = re.sub(r"[^0-9a-zA-Z]+", "_", torch.__version__)
    return os.path.join(BUILD, "_pgd_tensors_torch_%s.so" % tag)


def _older(path: str, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps)


def _library_stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER, __file__])


def _tensors_stale() -> bool:
    return _has_torch() and _older(tensors_path(), [TENSORS_SRC, HEADER, __file__])


def _torch_flags():
    """Compile and link flags of an extension against the installed torch."""
    import torch

    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api",
                                                     "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    lib = os.path.join(at, "lib")
    return (["-D_GLIBCXX_USE_CXX11_ABI=%d" % abi] + [x for p in inc for x in ("-isystem", p)],
            ["-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
             "-Wl,-rpath," + lib])


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if src == TENSORS_SRC:
        cmd = [os.environ.get("CXX", "g++")] + CXX_FLAGS + _torch_flags()[0] + ["-c", src, "-o", obj]
    elif src.endswith(".cu"):
        cmd = [_nvcc()] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + \
            ["-c", src, "-o", obj]
    else:
        cmd = [os.environ.get("CXX", "g++")] + CXX_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s\n%s" % (" ".join(cmd), r.stdout, r.stderr))
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libpgd.so, and the tensor extension where torch is
    installed; return the library's path."""
    force = force or verbose_ptxas
    library = sources() if force or _library_stale() else []
    tensors = [TENSORS_SRC] if (force and _has_torch()) or _tensors_stale() else []
    if not library and not tensors:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    jobs = tensors + library
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        objs = [ex.submit(_compile, s, verbose_ptxas) for s in jobs]
    # (the library first: it stands whatever becomes of the extension)
    if library:
        _link([_nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC"] +
              [o.result() for o in objs[len(tensors):]], LIB)
    if tensors:
        _link([os.environ.get("CXX", "g++"), "-shared", objs[0].result(), "-L" + BUILD, "-lpgd",
               "-Wl,-rpath,$ORIGIN"] + _torch_flags()[1], tensors_path())
    return LIB


def _link(cmd, path: str) -> None:
    tmp = path + ".tmp.%d" % os.getpid()
    cmd = cmd + ["-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed: %s\n%s\n%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, path)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
