"""Build libpkd.so (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc.

Translation units compile in parallel; the shared library links the CUDA runtime statically,
so it needs nothing at run time beyond the NVIDIA driver.  Output:
``paged_kv_decode_23_gb300/_build/libpkd.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpkd.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["decode_f16.cu", "decode_bf16.cu", "decode_e4m3.cu", "decode_rope.cu",
           "decode_rope_cc.cu", "decode_rope_cc_e4m3.cu", "mla.cu",
           "decode_sinks_rope_cc.cu", "decode_sinks_rope_cc_e4m3.cu", "decode_sinks_cc.cu",
           "decode_e2m1.cu", "decode_sinks.cu", "decode_scores.cu", "decode_e2m1_sinks.cu",
           "decode_e2m1_scores.cu", "key_weights.cu", "cache_append.cu", "cache_gather.cu", "cache_evict.cu",
           "cache_copy.cu", "cache_api.cpp",
           "mla_tc.cu", "planner.cpp", "pkd_api.cpp", "noalloc.cu"]
HEADERS = ["pkd_internal.h", "pkd_device.cuh", "decode_kernels.cuh", "decode_geometries.cuh",
           "decode_e2m1_kernels.cuh", "cache_ops.cuh", "cache_rows.cuh",
           "mla_kernels.cuh", "mla_tc_kernels.cuh"]


def _nvcc() -> str:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkd")
    return nvcc


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "pkd.h"))
    deps.append(os.path.abspath(__file__))
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(deps):
        return LIB
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3",
                     "-I", os.path.join(os.path.dirname(HERE), "include")]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
