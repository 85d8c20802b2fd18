"""Build liboidnx.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_calls.abi3.so, the binding's faster entry of the per-token calls (not needed: without
a C compiler or Python's headers the binding does without it).

Usage: python conv2d_implicit_gemm_gb300/build.py   (run as a script: importing the
package would load the library it is about to rebuild)

Translation units compile in parallel; the result is
conv2d_implicit_gemm_gb300/liboidnx.so.  Nothing here is imported at run time.
"""

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liboidnx.so")
CALLS = os.path.join(PKG, "_calls.abi3.so")  # the stable ABI: for any interpreter from 3.10 on
SOURCES = ["oidnx_host.cpp", "conv_tc.cu", "conv_pair.cu", "conv_final.cu", "conv_tail.cu",
           "conv_head.cu", "io_passes.cu", "noalloc.cu", "token_host.cpp", "linear_tc.cu", "linear_split.cu", "linear_align.cu",
           "qk_norm_rope.cu", "attn_any.cu", "attn_token.cu", "attn_prompt.cu", "attn_prompt64.cu",
           "block_host.cpp", "block_norm.cu", "cross_tile.cu", "cross_token.cu", "heads_copy.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def _nvcc():
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", path, "-o", obj]
    if src.endswith(".cpp"):
        cmd[cmd.index(path):cmd.index(path)] = ["-x", "cu"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
        results = list(pool.map(_compile, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=liboidnx.so", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _build_calls()
    return LIB


def _build_calls():
    """The Python entry of the per-token calls, linked to the library beside it; False if it cannot be built."""
    for stale in (CALLS, os.path.join(PKG, "_calls.so")):
        if os.path.exists(stale):
            os.remove(stale)
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC, "calls.c"), "-o", tmp, LIB, "-Wl,-rpath,$ORIGIN"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        failed = f"status {res.returncode}\n{res.stdout}{res.stderr}" if res.returncode else ""
    except OSError as e:
        failed = str(e)
    if failed:
        sys.stderr.write(f"{os.path.basename(CALLS)} could not be built, the per-token calls go through ctypes:\n{failed}\n")
        return False
    os.replace(tmp, CALLS)
    return True


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
