"""Builds libwtconv.so in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled in parallel into ``_build/`` and the
objects are linked into ``memory_bound_cnn_wtconv2d_gb300/libwtconv.so``
(the CUDA runtime is linked statically).  A rebuild happens only when a
source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libwtconv.so")
SOURCES = ("wtconv_api.cu", "wtconv_fwd.cu", "wtconv_fwd_win.cu", "wtconv_bwd_weight.cu", "wtconv_bwd_weight_win.cu",
           "wtconv_bwd_fused.cu", "wtconv_noalloc.cu", "wtconv_split.cu",
           # the operators around the layer (include/wtconv_block.h)
           "block/block_api.cu", "block/gn.cu", "block/gn_f32.cu", "block/gn_f16.cu", "block/gn_bf16.cu", "block/ns.cu",
           "block/ns_small.cu",
           # the gated channel mixer (include/wtconv_mixer.h)
           "block/mixer_api.cu", "block/rms.cu", "block/rms_f32.cu", "block/rms_f16.cu", "block/rms_bf16.cu", "block/clip.cu",
           "block/gated.cu", "block/gated_rows.cu")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwtconv")
    return path


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    for d in (CSRC, os.path.join(CSRC, "block")):
        files += glob.glob(os.path.join(d, "*.h")) + glob.glob(os.path.join(d, "*.cuh"))
    files += glob.glob(os.path.join(INCLUDE, "*.h"))
    return files


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            print(res.stdout + res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
