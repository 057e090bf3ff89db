"""Compile the CUDA sources into libmoe_pft.so (in-tree) for sm_103a with nvcc.

Each translation unit compiles in parallel into ``_build/``; the objects are linked into one
shared library next to this file.  Nothing is rebuilt when every object is newer than its
source and the headers.  ``csrc/marshal.cpp``, the binding's argument checks, becomes the Python
module ``_marshal.so`` beside it (host code; torch's headers), and is built again for another
Python or torch.
"""

from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_pft.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_KEY = os.path.join(BUILD, "marshal.txt")  # the Python and torch that MARSHAL was built for

SOURCES = ["api.cu", "gather.cu", "route.cu", "pft.cu", "pft_noalloc.cu", "gemm_simt.cu", "gemm_tc.cu", "router_tc.cu", "gshard.cu", "gemm_f32tc.cu",
           "norm.cu", "adamw.cu", "w4.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _headers():
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _marshal_key() -> str:
    import torch

    return f"python {sys.version}\ntorch {torch.__version__} {os.path.dirname(torch.__file__)}\n"


def _marshal_stale(source: str) -> bool:
    if _stale(MARSHAL, [source]) or not os.path.exists(MARSHAL_KEY):
        return True
    with open(MARSHAL_KEY) as f:
        return f.read() != _marshal_key()


def _marshal_command(source: str) -> list:
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            *[a for d in include for a in ("-isystem", d)], source, "-o", MARSHAL,
            "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False, force: bool = False, extra_flags=None) -> str:
    """Build (or reuse) libmoe_pft.so and return its path."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = _headers()
    extra = list(extra_flags or [])
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o])

    source = os.path.join(CSRC, "marshal.cpp")
    marshal = force or _marshal_stale(source)
    if marshal:
        jobs.insert(0, _marshal_command(source))

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed ({' '.join(cmd)}):\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    if marshal:
        with open(MARSHAL_KEY, "w") as f:
            f.write(_marshal_key())
    if force or _stale(LIB, objs):
        run([nvcc, *ARCH, "-shared", "-o", LIB, *objs])
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force="-f" in sys.argv,
          extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None)
    print(LIB)
