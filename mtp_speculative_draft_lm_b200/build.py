"""Builds the CUDA library ``libmtp.so`` in-tree for sm_100a (nvcc cross-compiles
without a GPU). Each ``csrc/*.cu`` becomes an object, rebuilt only when it or a
header changed; the objects are linked with the static CUDA runtime. Beside it, where
there is a torch, ``_block.so``, the module that makes the block cache's calls from torch
tensors: the library itself needs neither torch nor Python's headers."""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmtp.so")
CALLS_SRC = os.path.join(CSRC, "block_calls.cpp")
CALLS = os.path.join(PKG, "_block.so")
CALLS_KEY = os.path.join(BUILD, "block_calls.key")  # the torch and Python that CALLS was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest_dep = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj
    cmd = [NVCC, *ARCH, *CFLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _calls_key() -> str | None:
    """What _block.so is built for, found without importing torch; None where there is no torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"torch {version} at {os.path.dirname(spec.origin)}, Python {sys.version}"


def _build_calls(force: bool) -> None:
    key = _calls_key()
    if key is None:
        return
    newest = max(os.path.getmtime(f) for f in [CALLS_SRC, os.path.join(ROOT, "include", "mtp.h")])
    if not force and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= newest and os.path.exists(CALLS_KEY):
        with open(CALLS_KEY) as f:
            if f.read() == key:
                return
    import sysconfig

    import torch

    pkg = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(pkg, "include"),
           os.path.join(pkg, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(a for i in inc for a in ("-isystem", i)), CALLS_SRC, "-o", tmp,
           "-L" + os.path.join(pkg, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_KEY + f".tmp{os.getpid()}", "w") as f:
        f.write(key)
    os.replace(f.name, CALLS_KEY)


def _link(objs: list[str]) -> None:
    if os.path.exists(LIB) and os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs):
        return
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        calls = ex.submit(_build_calls, force)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        _link(objs)
        calls.result()  # (raises what went wrong with it: the library is there by now)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="--force" in sys.argv))
