"""Build libcsa2.so in-tree with nvcc for sm_103a (no cmake, no torch build).

``python -m compressed_sparse_attention_fp4_gb300.build`` compiles every
``csrc/*.cu`` in parallel and links ``_build/libcsa2.so``.  A rebuild is
skipped while the library is newer than every source and header.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libcsa2.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcsa2.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


# kernels whose roles share out the registers of the launch: source, its constant, their names
ROLE_SPLITS = {"dense.cu": ("kLaunchRegs", "dense_kernel|dense_pair_kernel"), "window.cu": ("kWinRegs", "window_kernel")}


def check_registers(source: str, ptxas: str, file: str = "dense.cu"):
    """Raises where ptxas gave a kernel of `file` (the dense attention's, the window attention's) another
    number of registers than the split among its roles counts on (the constant in `source`): the library
    would refuse every call, without this reason."""
    constant, kernels = ROLE_SPLITS[file]
    want = int(re.search(rf"{constant} = (\d+)", source).group(1))
    for name, got in re.findall(rf"entry function '\w*?\d({kernels})[EI]\w*'.*?Used (\d+) registers", ptxas, re.S):
        if int(got) != want:
            raise RuntimeError(f"{name}: {got} registers a thread, but its role split (csrc/{file}) is for {want}: "
                               f"build with the CUDA toolkit it was written for, or change {constant} and the split")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, "-Xptxas=-v", *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        if os.path.basename(src) in ROLE_SPLITS:
            with open(src) as f:
                check_registers(f.read(), r.stderr, os.path.basename(src))
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-lpthread", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
