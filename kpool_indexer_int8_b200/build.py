"""Build libglm_dsa.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python kpool_indexer_int8_b200/build.py [--force] [--verbose]

Each csrc/*.cu is compiled to an object under _build/ (rebuilt when it or a header changed) and
linked into kpool_indexer_int8_b200/libglm_dsa.so with the CUDA runtime linked statically.
csrc/args.c, the binding's checks of tensors, becomes kpool_indexer_int8_b200/_args.so (gcc, the headers
of this Python and the DLPack header that torch ships); where they are missing it is left out, with a
note, and the binding checks in Python.
No fast-math: the int8 quantisation relies on IEEE fp32 division and round-half-to-even.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libglm_dsa.so")
ARGS_SRC, ARGS_LIB = os.path.join(CSRC, "args.c"), os.path.join(PKG, "_args.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    extra = ["-Xptxas", "-v"] if verbose else []
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def build_args(force: bool = False) -> str:
    if force or not os.path.exists(ARGS_LIB) or os.path.getmtime(ARGS_LIB) < os.path.getmtime(ARGS_SRC):
        import importlib.util
        spec = importlib.util.find_spec("torch")
        if spec is None:
            raise RuntimeError("torch, whose DLPack header it needs, is not installed")
        torch = os.path.dirname(spec.origin)
        cmd = [os.environ.get("CC", "gcc"), "-O2", "-Wall", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
               "-I", os.path.join(torch, "include"), ARGS_SRC, "-o", ARGS_LIB + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {ARGS_SRC}:\n{r.stdout}\n{r.stderr}")
        os.replace(ARGS_LIB + ".tmp", ARGS_LIB)
    return ARGS_LIB


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    try:
        build_args(force)
    except (RuntimeError, OSError) as e:
        if os.path.exists(ARGS_LIB):
            os.remove(ARGS_LIB)                            # (of older sources)
        print(f"_args.so is not built, the binding checks its tensors in Python: {e}", file=sys.stderr)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hm = _headers_mtime()
    todo = []
    for s in srcs:
        obj = os.path.join(BUILD, os.path.basename(s) + ".o")
        if force or verbose or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(s), hm):
            todo.append(s)
    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(todo)))) as ex:
        list(ex.map(lambda s: _compile(s, verbose), todo))
    objs = [os.path.join(BUILD, os.path.basename(s) + ".o") for s in srcs]
    if todo or force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs,
               "-o", LIB + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
