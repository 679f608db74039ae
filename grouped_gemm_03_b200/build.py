"""Build libmoe.so (the C-ABI library) in-tree with nvcc for sm_100a, and _ops.so
beside it, the compiled part of the Python binding (g++, PyTorch's headers; left
out where PyTorch is not installed, and built again when it is another one).

    python -m grouped_gemm_03_b200.build [--force] [-v]
    python grouped_gemm_03_b200/build.py                 # the same, without importing PyTorch for the C library

Objects go to _build/ at the repository root; the shared library lands next
to this file so the Python binding finds it.  cudart is linked statically, so
the library needs only the NVIDIA driver at run time.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmoe.so")
OPS_SRC = os.path.join(CSRC, "binding", "ops.cpp")
OPS = os.path.join(HERE, "_ops.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, obj: str, extra: list[str], verbose: bool) -> None:
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdr = _headers_mtime()
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        stale = force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr)
        if stale:
            jobs.append((src, obj))
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        for f in [ex.submit(_compile, s, o, extra, verbose) for s, o in jobs]:
            f.result()
    if jobs or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_ops(force, verbose)
    return LIB


def _ops_made_for() -> str | None:
    """What _ops.so is compiled against: PyTorch and Python, where PyTorch is there (None: it is not)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    return f"torch {importlib.metadata.version('torch')} at {spec.origin}, python {sys.version}"


def _build_ops(force: bool, verbose: bool) -> None:
    header, stamp = os.path.join(INCLUDE, "moe.h"), os.path.join(BUILD, "ops.made_for")
    made_for = _ops_made_for()
    if made_for is None:   # the C library is complete without the Python binding
        if verbose:
            print("no PyTorch: _ops.so (the Python binding's compiled part) is not built", flush=True)
        return
    known = None
    if os.path.exists(stamp):
        with open(stamp) as f:
            known = f.read()
    if (not force and known == made_for and os.path.exists(OPS) and
            os.path.getmtime(OPS) >= max(map(os.path.getmtime, (OPS_SRC, header)))):
        return
    import torch

    at = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    includes = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"), cuda,
                INCLUDE, sysconfig.get_paths()["include"]]
    tmp = OPS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{d}" for d in includes), OPS_SRC,
           "-o", tmp, f"-L{os.path.join(at, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python", f"-L{HERE}", "-l:libmoe.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(OPS_SRC)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS)
    with open(stamp, "w") as f:
        f.write(made_for)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args(argv)
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, ptxas_info=a.ptxas_info))
    return 0


if __name__ == "__main__":
    sys.exit(main())
