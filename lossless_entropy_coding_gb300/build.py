"""Build the CUDA library in-tree: nvcc for sm_103a, one translation unit per
process, linked into lossless_entropy_coding_gb300/_build/libecc_gb300.so.
build(checked=True) builds the index-checked variant (-DECC_CHECKED: the
kernels test their shared- and global-memory indices, skip an access out of
range and report ECC_ERR_CHECK) into _build_checked/libecc_gb300_checked.so.
build_torch() builds the Python module that unpacks torch tensors for the
language-model operators (g++, torch's headers) into _build/ecc_torch.so.

    python -m lossless_entropy_coding_gb300.build [--force] [--checked]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libecc_gb300.so")
CHECKED_DIR = os.path.join(HERE, "_build_checked")
CHECKED_LIB = os.path.join(CHECKED_DIR, "libecc_gb300_checked.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in ("ecc.h", "ecc_lm.h")]
    return files


def _compile(src: str, nvcc: str, extra, out_dir: str = OUT_DIR) -> str:
    obj = os.path.join(out_dir, os.path.basename(src) + ".o")
    cmd = [nvcc, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
           *extra, "-c", src, "-o", obj]
    subprocess.check_call(cmd)
    return obj


def build(force: bool = False, extra=(), checked: bool = False) -> str:
    out_dir, lib = (CHECKED_DIR, CHECKED_LIB) if checked else (OUT_DIR, LIB)
    flags = list(extra) + (["-DECC_CHECKED"] if checked else [])
    os.makedirs(out_dir, exist_ok=True)
    newest = max(os.path.getmtime(f) for f in _deps())
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= newest:
        return lib
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=len(sources())) as ex:
        objs = list(ex.map(lambda s: _compile(s, nvcc, flags, out_dir), sources()))
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"])
    os.replace(tmp, lib)
    return lib


TORCH_LIB = os.path.join(OUT_DIR, "ecc_torch.so")


def build_torch(force: bool = False) -> str:
    """After build(): the module links against the library."""
    import torch

    src = os.path.join(CSRC, "torch", "ecc_torch.cpp")
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(INCLUDE, "ecc_lm.h"), os.path.join(INCLUDE, "ecc.h")))
    if not force and os.path.exists(TORCH_LIB) and os.path.getmtime(TORCH_LIB) >= newest:
        return TORCH_LIB
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    subprocess.check_call([
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-I", INCLUDE, "-I", os.path.join(home, "include"), "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
        "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"], src, "-o", tmp,
        "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
        f"-Wl,-rpath,{os.path.join(home, 'lib')}", "-L", OUT_DIR, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, TORCH_LIB)
    return TORCH_LIB


def main(argv) -> None:
    force, checked = "--force" in argv, "--checked" in argv
    print(build(force=force, checked=checked))
    if checked:
        return
    try:
        print(build_torch(force=force))
    except ImportError:
        print("PyTorch is not installed: the library is built, ecc_torch (the Python entry points of the "
              "language-model operators) is not", file=sys.stderr)


if __name__ == "__main__":
    main(sys.argv[1:])
