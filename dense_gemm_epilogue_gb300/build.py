"""Build the tg_gemm shared library for sm_103a with nvcc (no GPU needed).

Each translation unit compiles in its own process, in parallel, then one
link step writes ``_lib/libtg_gemm.so`` next to this file (in-tree, so that
the library the tests and the benchmark load is the one built here).
"""

from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libtg_gemm.so")
PYCALL_SOURCE = os.path.join(CSRC, "tg_pycall.c")
# (an extension module belongs to one interpreter version: its name says which)
PYCALL = os.path.join(OUT_DIR, "_tgcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
OBJ_DIR = os.path.join(HERE, "_build")
SOURCES = ["tg_gemm.cu", "tg_inst_bf16.cu", "tg_inst_fp16.cu", "tg_inst_tf32.cu",
           "tg_inst_e4m3.cu", "tg_inst_e5m2.cu", "tg_inst_mx.cu", "tg_noalloc.cu", "tg_mlp.cu",
           "tg_norm.cu", "tg_inst_mlp_bf16_cg1.cu", "tg_inst_mlp_bf16_cg2.cu",
           "tg_inst_mlp_fp16_cg1.cu", "tg_inst_mlp_fp16_cg2.cu", "tg_inst_stream_bf16.cu",
           "tg_inst_stream_fp16.cu", "tg_rotary.cu", "tg_attn.cu", "tg_inst_attn_bf16.cu",
           "tg_inst_attn_fp16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


# What the dense GEMM's kernels are compiled from and planned by.
GEMM_SOURCES = ["tg_gemm.cu", "tg_inst.cuh", "tg_inst_bf16.cu", "tg_inst_e4m3.cu", "tg_inst_e5m2.cu",
                "tg_inst_fp16.cu", "tg_inst_tf32.cu", "tg_kernel.cuh", "tg_kernel_mx.cuh",
                "tg_kernel_pair.cuh", "tg_launch.h", "tg_ptx.cuh"]


def _hash(paths) -> str:
    h = hashlib.sha256()
    for p in paths:
        with open(p, "rb") as f:
            h.update(os.path.basename(p).encode() + b"\0" + f.read())
    return h.hexdigest()[:16]


def source_hash() -> str:
    """Hash of every kernel/host source and header (identifies a build)."""
    names = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h")))
    return _hash([os.path.join(CSRC, n) for n in names] + [os.path.join(ROOT, "include", "tg_gemm.h")])


def gemm_source_hash() -> str:
    """Hash of the dense GEMM's sources alone: a figure measured on its kernels
    holds while this one does, whatever the other operators' sources become."""
    return _hash([os.path.join(CSRC, n) for n in GEMM_SOURCES])


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _build_pycall(force: bool) -> None:
    """The host-only module that marshals the hot Python calls, with a stamp of
    its own beside it.  Without Python's headers or a C compiler the ctypes
    wrappers serve alone, and the next build() looks again; what the compiler
    refuses (an old Python's headers, say) costs a warning, not the library."""
    stamp = PYCALL + ".hash"
    want = _hash([PYCALL_SOURCE, os.path.join(ROOT, "include", "tg_gemm.h")])
    if not force and os.path.exists(PYCALL) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == want:
                return
    for old in (PYCALL, stamp):
        if os.path.exists(old):
            os.remove(old)
    include = sysconfig.get_paths()["include"]
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None or not os.path.exists(os.path.join(include, "Python.h")):
        return
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = PYCALL + ".tmp.%d" % os.getpid()
    r = subprocess.run([cc, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", "-I", include, "-I",
                        os.path.join(ROOT, "include"), PYCALL_SOURCE, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        warnings.warn(f"{cc} failed on tg_pycall.c, calls go through ctypes:\n{r.stdout}\n{r.stderr}",
                      RuntimeWarning, stacklevel=3)
        return
    os.replace(tmp, PYCALL)
    with open(stamp, "w") as f:
        f.write(want + "\n")


def _build_library(force: bool, verbose_ptxas: bool) -> None:
    stamp = os.path.join(OUT_DIR, "BUILD_HASH")
    want = source_hash()
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == want:
                return
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(want + "\n")


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    _build_library(force, verbose_ptxas)
    _build_pycall(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
