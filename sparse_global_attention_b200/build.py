"""Build the GSA shared library (libgsa_b200.so) in-tree with nvcc for sm_100a.

    python -m sparse_global_attention_b200.build [--debug]

Each .cu under csrc/ compiles to an object in _build/ (in parallel); the
objects link into sparse_global_attention_b200/libgsa_b200.so.  Only the CUDA
runtime is linked (statically, so the library needs nothing at run time but the
driver).  csrc/torch_binding.cpp, the marshalling of torch tensors for the
operators around the layer, becomes _torch_binding.so beside it (host code
against the installed torch's headers; it has no kernels).  The library does not
depend on it: without torch the C ABI is built and a message says what is missing,
and a binding that does not compile is reported once the library is there.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgsa_b200.so")
BINDING = os.path.join(PKG, "_torch_binding.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for p in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if p and os.path.exists(p):
            return p
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgsa_b200.so")


def build_binding() -> str:
    """Compile the binding; ImportError where torch (or what its extension tools need) is not installed."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    libs = cpp_extension.library_paths()
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for d in inc for a in ("-isystem", d)], os.path.join(CSRC, "torch_binding.cpp"), "-o", tmp,
           *[f"-L{d}" for d in libs], "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_binding.cpp:\n{r.stdout}\n{r.stderr}")
    if r.stderr:
        sys.stderr.write(r.stderr)
    os.replace(tmp, BINDING)
    return BINDING


def build(debug: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    flags = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC] + ARCH
    if debug:
        flags += ["-DGSA_DEBUG=1"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objs = []

    def one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc(), *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = ex.submit(build_binding)
        for obj, log in ex.map(one, srcs):
            objs.append(obj)
            if verbose and log:
                sys.stderr.write(log)
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        try:
            binding.result()
        except ImportError as e:
            sys.stderr.write(f"{os.path.basename(LIB)} is built; {os.path.basename(BINDING)}, which the Python operators "
                             f"around the layer need, is not, since torch's extension tools are not there: {e}\n")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--debug", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args()
    print(build(debug=args.debug, verbose=args.verbose))
