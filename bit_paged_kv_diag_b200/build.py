"""Build libkvq.so (the C-ABI library and its sm_100a kernels) in-tree.

    python -m bit_paged_kv_diag_b200.build        # or: python bit_paged_kv_diag_b200/build.py

nvcc cross-compiles for sm_100a without a GPU.  The library is written next to this
file, so it travels with the source tree.
"""
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvq.so")
SOURCES = ["kvq_api.cu", "append_kernel.cu", "decode_kernel.cu", "kvq_noalloc.cu",
           "prefill_tc.cu", "kvq_ops.cu", "rope_append.cu", "gather_rows.cu", "block_bounds.cu",
           "block_select.cu", "sparse_attention.cu"]
HEADERS = ["kvq_internal.h", "kvq_ptx.cuh", "append_row.cuh", "decode_tile.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "kvq.h"))
    return files


def build(force: bool = False, verbose: bool = False) -> str:
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(f) for f in _inputs())):
        return LIB
    # One object per source, compiled side by side, then one link.
    objs = tempfile.mkdtemp(prefix="kvq_build_")
    tmp = LIB + f".tmp{os.getpid()}"
    verbose_flags = ["-Xptxas=-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(objs, src + ".o")
        subprocess.run([_nvcc(), *verbose_flags, *NVCC_FLAGS, "-c", "-o", obj, os.path.join(CSRC, src)],
                       check=True)
        return obj

    try:
        with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as ex:
            done = list(ex.map(compile_one, SOURCES))
        subprocess.run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *done], check=True)
        os.replace(tmp, LIB)
    finally:
        shutil.rmtree(objs, ignore_errors=True)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
