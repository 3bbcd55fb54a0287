"""Build libwkv_b200.so in-tree with nvcc for sm_100a (B200).

    python -m linear_attention_rnn_wkv_b200.build [--verbose]

The library is a plain C ABI (include/wkv.h); it links the shared CUDA runtime so it
shares one runtime instance with PyTorch in the same process.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libwkv_b200.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "shared",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in sources() + headers() + [__file__])


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    common = [nvcc()] + NVCC_FLAGS + ["-I", INCLUDE, "-I", CSRC]
    # the sources compile side by side, then one link
    with tempfile.TemporaryDirectory() as objs:
        steps = [common + (["-Xptxas", "-v"] if ptxas_info else []) +
                 ["-c", src, "-o", os.path.join(objs, os.path.basename(src) + ".o")] for src in sources()]
        with concurrent.futures.ThreadPoolExecutor(os.cpu_count()) as pool:
            done = list(pool.map(lambda cmd: (cmd, subprocess.run(cmd, capture_output=True, text=True)), steps))
        if all(res.returncode == 0 for _, res in done):
            link = common + [cmd[-1] for cmd in steps] + ["-o", tmp]
            done.append((link, subprocess.run(link, capture_output=True, text=True)))
    for cmd, res in done:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            print(res.stdout + res.stderr, file=sys.stderr)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
