"""Build libmars.so in-tree with nvcc for sm_103a (one -gencode, translation units
compiled in parallel, no cmake), and the C form of packed.py's calls. `python -m block_masked_token_gb300.build` or
`build_library()`."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmars.so")
CALLS = os.path.join(PKG, "_packed_calls" + sysconfig.get_config_var("EXT_SUFFIX"))

SOURCES = ["mars_api.cu", "kv_commit.cu", "decode_attn.cu", "head_accept.cu", "dual_stream.cu",
           "tmap.cu", "head_accept_noalloc.cu", "ce_loss.cu", "dual_stream_grad.cu",
           "packed_attn.cu", "packed_grad.cu", "kv_append.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmars")
    return exe


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _build_calls() -> None:
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        raise RuntimeError("gcc not found: it is required to build packed.py's calls")
    tmp = CALLS + ".tmp"
    cmd = [cc, "-O2", "-Wall", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I",
           os.path.join(ROOT, "include"), os.path.join(CSRC, "packed_calls.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on packed_calls.c:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def build_library(verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        calls = ex.submit(_build_calls)
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
        calls.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library(verbose_ptxas="-v" in sys.argv))
