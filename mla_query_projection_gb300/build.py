"""Build ``libmla_query.so`` (the C-ABI library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into one
shared library next to this file.  The CUDA runtime is linked statically, so
the library loads on a machine without a GPU (every call then returns
MLA_ECUDA).  ``csrc/torch/tensor_calls.cpp``, the module through which torch
tensors reach the cache-side operators, is compiled by the host compiler into
``_tensor_calls.so`` beside it (where that fails, the library is built all the
same, and the failure raised).  Usage: ``python -m mla_query_projection_gb300.build``.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmla_query.so")
BUILD = os.path.join(HERE, "_build")
CALLS_SRC = os.path.join(CSRC, "torch", "tensor_calls.cpp")
CALLS = os.path.join(HERE, "_tensor_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3",
    "-lineinfo",
    "-std=c++17",
    "-Xcompiler",
    "-fPIC",
    "-Xcompiler",
    "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-Xptxas",
    "-v",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla_query.so")
    return cand


def _compile(src: str, build_dir: str = BUILD, extra: tuple = ()) -> tuple[str, str]:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{p.stdout}\n{p.stderr}")
    return obj, p.stderr


def _compile_calls() -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed: _tensor_calls.so, which it needs, is not built")
    torch = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(torch, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", *("-I" + i for i in include),
           CALLS_SRC, "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-o", tmp]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, CALLS)


def build(verbose: bool = False, out_dir: str | None = None, extra: tuple = ()) -> str:
    """Compile and link; returns the path of the shared library.  With
    `out_dir` and `extra` nvcc flags, a variant of the same sources goes into
    out_dir (for instance the bounds-checked build, extra=("-DMLA_CHECKS",));
    the in-tree library is left as it is."""
    build_dir = BUILD if out_dir is None else out_dir
    lib = LIB if out_dir is None else os.path.join(out_dir, "libmla_query.so")
    os.makedirs(build_dir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_compile_calls) if out_dir is None else None
        results = list(ex.map(lambda src: _compile(src, build_dir, tuple(extra)), srcs))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, lib)
    with open(os.path.join(build_dir, "ptxas.log"), "w") as f:
        for _, log in results:
            f.write(log)
    if calls is not None:
        calls.result()  # (a failure is raised here: the C library stands without the module)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
