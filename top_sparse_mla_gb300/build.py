"""Compile the CUDA library (libdsa_sparse_attn.so) in-tree for sm_103a."""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SOURCES = [os.path.join(PKG_DIR, "csrc", f) for f in ("dsa_sparse_attn.cu", "dsa_kv8_attn.cu", "dsa_kv8_tiles.cu",
                                                      "dsa_kv8_insert.cu", "dsa_topk.cu", "dsa_kv_insert.cu", "dsa_page_map.cu")]
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libdsa_sparse_attn.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")


def build(verbose: bool = False, extra_flags=None) -> str:
    """Build the shared library if any source is newer than it; return its path.  The
    sources are compiled at the same time, one nvcc each, and then linked."""
    csrc = os.path.join(PKG_DIR, "csrc")
    headers = [os.path.join(where, h) for where in (INCLUDE, csrc) for h in sorted(os.listdir(where)) if h.endswith((".h", ".cuh"))]
    deps = SOURCES + headers + [os.path.abspath(__file__)]
    if os.path.exists(LIB_PATH) and all(os.path.getmtime(LIB_PATH) >= os.path.getmtime(d) for d in deps):
        return LIB_PATH
    flags = [*ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, *(extra_flags or [])]
    nvcc = nvcc_path()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    with tempfile.TemporaryDirectory(prefix="dsa_build_") as objs:
        jobs = [(src, os.path.join(objs, os.path.basename(src) + ".o")) for src in SOURCES]
        with ThreadPoolExecutor(len(jobs)) as pool:
            list(pool.map(lambda job: _run([nvcc, *flags, "-c", "-o", job[1], job[0]], verbose), jobs))
        _run([nvcc, *ARCH_FLAGS, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *[obj for _, obj in jobs], *(extra_flags or [])],
             verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
