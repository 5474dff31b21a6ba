"""In-tree build of ``libflce.so`` for sm_103a with nvcc (no cmake, no setuptools), and of ``flce_torch``, the
native marshalling of torch tensors, with the host compiler.

The translation units compile in parallel; each output is rebuilt only when a
source or header is newer than it is.  The library does not depend on the
marshalling: it is linked also where that does not compile, which is then
raised.  Output: ``linear_cross_entropy_tmem_gb300/_build/``.

    python -m linear_cross_entropy_tmem_gb300.build
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

from .binding import torch_path

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libflce.so")
SOURCES = ["flce_api.cu", "flce_fwd.cu", "flce_bwd.cu", "flce_noalloc.cu", "flce_norm.cu", "flce_norm_fwd.cu",
           "flce_norm_fp8.cu", "flce_norm_fp8_left.cu", "flce_norm_bwd.cu", "flce_clip.cu", "flce_logits.cu"]
TORCH_SOURCE = "flce_torch.cpp"
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libflce.so")


def _flags():
    return [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
            f"-I{INCLUDE}", f"-I{CSRC}"]


def _stale(output: str) -> bool:
    """Whether ``output`` is missing or older than a source or header."""
    files = glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    files.append(os.path.abspath(__file__))
    return not os.path.exists(output) or os.path.getmtime(output) < max(os.path.getmtime(f) for f in files)


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_torch(out: str) -> None:
    """flce_torch: a Python extension on torch's C++ interface."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}", f"-isystem{inc}",
           f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-isystem{cuda}",
           f"-I{sysconfig.get_paths()['include']}", os.path.join(CSRC, TORCH_SOURCE), "-o", tmp, f"-L{lib}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {TORCH_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    cmd = [nvcc(), ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build (or reuse) libflce.so and flce_torch, and return the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    torch_lib = torch_path()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_torch, torch_lib) if force or _stale(torch_lib) else None
        if force or _stale(LIB):
            _link(list(ex.map(_compile, SOURCES)))
            if verbose:
                print(f"built {LIB}")
        if marshal is not None:
            marshal.result()
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
