"""Build libgnn_spmm.so (HIP, gfx950) in-tree with hipcc, and _rows.so with g++.

Each translation unit under csrc/ is compiled separately (in parallel) and the
objects are linked into gnn_sparse_dense_amd/libgnn_spmm.so next to this file.
_rows.so holds the row operators' torch autograd nodes: host code that calls
the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgnn_spmm.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = [
    "api.cpp",
    "alloc.cpp",
    "plan_kernels.hip",
    "combine.hip",
    "row_kernels_v1.hip",
    "row_kernels_v2.hip",
    "row_kernels_v4.hip",
    "window_kernels.hip",
    "transform.hip",
    "mfma_tile.hip",
    "features.hip",
    "pair_kernel.hip",
    "reorder.hip",
    "merge_kernel.hip",
    "split_fused.hip",
    "exchange.hip",
    "layer_norm.hip",
    "segment.hip",
]

COMMON = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    "-Wall",
    "-Wno-unused-result",
    # no packed fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE fp32 division for the mean (also hipcc's default; stated explicitly)
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-fast-math",
    f"-I{os.path.join(ROOT, 'include')}",
]


def _compile(src: str) -> str:
    out = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") or src.endswith(".cpp") else []
    cmd = [HIPCC, *COMMON, *lang, "-c", os.path.join(CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return out


ROWS = os.path.join(HERE, "_rows.so")


def _compile_rows() -> str:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    out = os.path.join(OBJ, "torch_rows.o")
    includes = [*include_paths(), os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
                sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-sign-compare",
           "-DTORCH_EXTENSION_NAME=_rows", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-isystem{p}" for p in includes], "-c", os.path.join(CSRC, "torch_rows.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_rows.cpp:\n{r.stdout}\n{r.stderr}")
    return out


def _link_rows(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = ROWS + ".tmp"
    cmd = ["g++", "-shared", obj, "-o", tmp, f"-L{HERE}", "-lgnn_spmm", f"-L{libs}", "-lc10", "-lc10_hip",
           "-ltorch", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ROWS)


def build(verbose: bool = True, jobs: int = 8) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        rows = ex.submit(_compile_rows)
        objs = list(ex.map(_compile, SOURCES))
        rows = rows.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_rows(rows)
    if verbose:
        print(f"built {LIB} and {ROWS}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
