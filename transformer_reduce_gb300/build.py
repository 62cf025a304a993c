"""Build libls_reduce.so in-tree with nvcc for sm_103a (GB300).

One translation unit per storage dtype plus the ABI layer, compiled in
parallel, then linked into a shared library with the CUDA runtime linked
statically (the library depends on nothing but the driver).  The result is
written next to this file and loaded by ``transformer_reduce_gb300._lib``.

    python -m transformer_reduce_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libls_reduce.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

SOURCES = ["abi.cu", "kernels_f32.cu", "kernels_f16.cu", "kernels_bf16.cu", "noalloc.cu",
           "cross_entropy.cu", "linear_ce.cu",
           "diff_fw_f32.cu", "diff_fw_f16.cu", "diff_fw_bf16.cu", "diff_bw_f32.cu", "diff_bw_f16.cu",
           "diff_bw_bf16.cu", "block_norm_fw_f32.cu", "block_norm_fw_f16.cu",
           "block_norm_fw_bf16.cu", "block_norm_bw_f32.cu", "block_norm_bw_f16.cu",
           "block_norm_bw_bf16.cu", "relpos_fw_f32.cu", "relpos_fw_f16.cu",
           "relpos_fw_bf16.cu", "relpos_bw_f32.cu", "relpos_bw_f16.cu", "relpos_bw_bf16.cu",
           "qk_norm_rope_f32.cu", "qk_norm_rope_f16.cu", "qk_norm_rope_bf16.cu", "grad_clip.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libls_reduce.so")
    return cand


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "ls_reduce.h"))
    files.append(os.path.abspath(__file__))
    return files


def _up_to_date(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
           os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose:
        sys.stderr.write(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and link libls_reduce.so; return its path."""
    deps = _deps()
    if not force and not verbose and _up_to_date(LIB_PATH, deps):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register / spill report")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
