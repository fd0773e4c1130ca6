"""Build libmfa_gb300.so in-tree with nvcc for sm_103a (GB300), and _binding.so,
the CPython module of the short calls, against it and torch's headers.

Each translation unit is compiled in parallel, then linked into one shared
library and one module next to this file.  Nothing is installed anywhere.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmfa_gb300.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(BUILD, "built_for.txt")
SOURCES = ["api.cu", "sched.cu", "topk.cu", "decode.cu", "prefill_sm103.cu", "prefill_f16.cu", "backward.cu", "backward_sm103.cu", "noalloc.cu", "rope.cu", "chunk.cu", "chunk_sm103.cu",
           "chunk_f16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmfa_gb300.so")
    return cand


def torch_dir() -> str:
    spec = importlib.util.find_spec("torch")  # found, not imported
    if spec is None:
        raise RuntimeError("torch not found: the binding is compiled against its headers")
    return os.path.dirname(spec.origin)


def torch_version() -> str:
    """torch.__version__, read without importing torch."""
    with open(os.path.join(torch_dir(), "version.py")) as f:
        return re.search(r"__version__ = ['\"](.*?)['\"]", f.read()).group(1)


def _deps_mtime() -> float:
    m = 0.0
    for d in (CSRC, os.path.join(ROOT, "include")):
        for f in os.listdir(d):
            m = max(m, os.path.getmtime(os.path.join(d, f)))
    return max(m, os.path.getmtime(__file__))


def built_for() -> str:
    """What the binding is compiled against, which no time of a source file tells."""
    return f"torch {torch_version()}, python {sysconfig.get_config_var('SOABI')}\n"


def stale() -> bool:
    outputs = (LIB, BINDING, BUILT_FOR)
    if not all(os.path.exists(f) for f in outputs) or min(map(os.path.getmtime, outputs)) < _deps_mtime():
        return True
    with open(BUILT_FOR) as f:
        return f.read() != built_for()


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile (if stale) and return the path of the shared library."""
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_verbose:
            print(r.stdout + r.stderr)
        return obj

    def compile_binding():
        obj = os.path.join(BUILD, "binding.o")
        include = [os.path.join(ROOT, "include"), os.path.join(torch_dir(), "include"),
                   os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include"),
                   sysconfig.get_paths()["include"]]
        run(["g++", "-O2", "-std=c++17", "-fPIC", f'-DMFA_TORCH_VERSION="{torch_version()}"', *("-I" + d for d in include), "-c",
             os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ failed for binding.cpp")
        return obj

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding_obj = binding.result()
    tmp = LIB + ".tmp"
    run([cc, *ARCH, "-shared", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB)
    # torch's libraries are those that `import torch` has loaded, the kernels' library is the one beside the module
    tmp = BINDING + ".tmp"
    run(["g++", "-shared", "-o", tmp, binding_obj, "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
         "-L" + os.path.join(torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"],
        "link of the binding failed")
    os.replace(tmp, BINDING)
    with open(BUILT_FOR, "w") as f:
        f.write(built_for())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
