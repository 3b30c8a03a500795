"""Build libtps.so (the CUDA library behind include/tps.h) in-tree.

Each translation unit in csrc/ is compiled by nvcc for sm_103a in parallel,
then linked into a shared library with the CUDA runtime linked statically,
so loading the library needs no GPU and no libcuda at load time (the driver
entry points are resolved through the runtime on first use).  Beside it the
CPython extension _binding.so (csrc/binding.cpp), the Python side of the
short calls, is compiled by the host compiler against the installed torch.

`debug=True` builds libtps_debug.so instead (TPS_DEBUG=1: every direct store
of the GEMMs' epilogues and of the vocabulary-sharded cross-entropy is checked
against the bounds of its output, and a store outside is skipped and reported
as TPS_ERR_BOUNDS, those of the linear product among them; the kernels around
the GEMMs of linear_ce.cu and linear.cu, rope.cu, optim.cu, norm.cu and
dropout.cu have no such check).  Set
TPS_LIBRARY to its path to make the Python binding load it.

    python -m backward_tcgen05_tma_gemms_gb300.build [--force] [--debug]
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtps.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_STAMP = os.path.join(PKG, "_build", "binding.txt")  # the torch that it was compiled against
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libtps_debug.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, extra, build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _torch_stamp() -> str:
    """What the extension is compiled against: it fits no other torch or Python."""
    import torch
    return f"{torch.__version__} {torch.version.git_version} {os.path.dirname(torch.__file__)} {sys.version}"


def _binding_current() -> bool:
    """Whether the extension is newer than the sources and was compiled against the installed torch."""
    try:
        with open(BINDING_STAMP) as f:
            return os.path.getmtime(BINDING) >= _deps_mtime() and f.read() == _torch_stamp()
    except OSError:
        return False


def _compile_binding() -> None:
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    os.makedirs(BUILD, exist_ok=True)
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(at, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           f"-Wl,-rpath,{os.path.join(at, 'lib')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stderr}")
    if os.path.exists(BINDING_STAMP):
        os.remove(BINDING_STAMP)
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_torch_stamp())


def build(force: bool = False, verbose_ptxas: bool = False, debug: bool = False) -> str:
    """Compile and link libtps.so (libtps_debug.so with debug=True) and the
    extension if any source is newer than they, the extension also if it was
    compiled against another torch; return the library's path."""
    lib, build_dir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _deps_mtime():
        if not _binding_current():
            _compile_binding()
        return lib
    os.makedirs(build_dir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    if debug:
        extra += ["-DTPS_DEBUG=1"]
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = None if not force and _binding_current() else ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, extra, build_dir), srcs))
        if binding is not None:
            binding.result()
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register / shared memory usage")
    ap.add_argument("--debug", action="store_true", help="build libtps_debug.so (bounds-checked stores)")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.ptxas_v, debug=a.debug))
