"""Build libadmmq.so (sm_100a) in-tree with nvcc.

    python -m post_weight_quantization_10_b200.build [--verbose]

The library is compiled for sm_100a only and links cuSOLVER (the one-time
eigendecomposition) from the CUDA toolkit.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libadmmq.so")
SOURCES = ["admmq.cu", "mx.cu", "packed.cu", "packed_gemm_bf16.cu", "packed_gemm_fp16.cu"]
HEADERS = ["host.cuh", "async.cuh", "gave_up.cuh", "ptx.cuh", "gemm.cuh", "kernels.cuh", "admm_loop.cuh", "gptq.cuh", "mx.cuh",
           "mx_gemm.cuh", "packed.cuh", "packed_few.cuh", "packed_gemm.cuh",
           "packed_gemm_launch.cuh", "tmem_fair.cuh"]
INCLUDE = os.path.join(os.path.dirname(HERE), "include", "admmq.h")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [INCLUDE]
    return any(os.path.getmtime(p) > t for p in deps)


def _run(cmd, verbose: bool) -> int:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stdout.write(res.stdout)
        sys.stderr.write(res.stderr)
    return res.returncode


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    cuda_home = os.path.dirname(os.path.dirname(nvcc))
    libdir = os.path.join(cuda_home, "lib64")
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]
    with tempfile.TemporaryDirectory(dir=HERE, prefix=".build_") as tmp:
        # the sources are compiled side by side, then linked
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        cmds = [[nvcc] + flags + ["-c", "-o", o, os.path.join(CSRC, s)]
                for s, o in zip(SOURCES, objs)]
        link = [nvcc] + flags + ["-shared", "-o", LIB + ".tmp"] + objs + [
            "-L" + libdir, "-lcusolver", "-lcublas", "-Xlinker", "-rpath," + libdir]
        with ThreadPoolExecutor(len(cmds)) as pool:
            for res in pool.map(lambda c: _run(c, verbose), cmds):
                if res:
                    raise RuntimeError(f"nvcc failed with exit code {res}")
        if _run(link, verbose):
            raise RuntimeError("linking failed")
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          ptxas_info="--ptxas" in sys.argv)
    print(LIB)
