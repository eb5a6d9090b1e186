"""Build and load the native library (libspec_verify.so, CUDA for sm_103a)."""
from __future__ import annotations

import concurrent.futures
import ctypes
import os
import subprocess
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", name) for name in ("spec_verify.cu", "spec_attn.cu")]
HEADERS = [os.path.join(ROOT, "include", name) for name in ("spec_verify.h", "spec_attn.h")] + [
    os.path.join(PKG, "csrc", name) for name in ("attn_common.cuh", "attn_plan.cuh", "attn_tile.cuh")]
LIB = os.path.join(PKG, "libspec_verify.so")
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC"]

_lock = threading.Lock()
_lib = None


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu, in parallel, into libspec_verify.so beside this file."""
    with _lock:
        stale = not os.path.exists(LIB) or any(
            os.path.getmtime(LIB) < os.path.getmtime(p) for p in (*SOURCES, *HEADERS))
        if force or stale:
            tmp = LIB + f".tmp{os.getpid()}"
            flags = [*NVCC_FLAGS, "-I", os.path.join(ROOT, "include")]
            if verbose:
                flags.append("-Xptxas=-v")
            objects = [f"{tmp}.{os.path.basename(src)}.o" for src in SOURCES]
            try:
                with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
                    list(ex.map(lambda so: subprocess.check_call([nvcc(), *flags, "-c", "-o", so[1], so[0]]),
                                zip(SOURCES, objects)))
                subprocess.check_call([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objects])
                os.replace(tmp, LIB)
            finally:
                for path in (tmp, *objects):
                    if os.path.exists(path):
                        os.remove(path)
    return LIB


def load() -> ctypes.CDLL:
    """Load the CUDA library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError(f"native library {LIB} is missing: build it with __graft_entry__.build() "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB)
    vp, i, u, p = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.POINTER
    lib.spec_verify_init.restype = i
    lib.spec_verify_init.argtypes = [p(vp), i, i, i, i, u]
    lib.spec_verify.restype = i
    lib.spec_verify.argtypes = [vp, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_verify_lazy.restype = i
    lib.spec_verify_lazy.argtypes = [vp, i, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_verify_loss_grad.restype = i
    lib.spec_verify_loss_grad.argtypes = [vp, i, vp, vp, vp, i, vp, vp, vp, vp]
    lib.spec_verify_ex.restype = i
    lib.spec_verify_ex.argtypes = [vp, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_verify_noalloc.restype = i
    lib.spec_verify_noalloc.argtypes = [i, i, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_verify_tv.restype = i
    lib.spec_verify_tv.argtypes = [vp, i, vp, vp, vp, vp, vp]
    lib.spec_verify_host.restype = i
    lib.spec_verify_host.argtypes = [vp, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_verify_get_error.restype = i
    lib.spec_verify_get_error.argtypes = [vp, p(i)]
    lib.spec_verify_selftest_wait.restype = i
    lib.spec_verify_selftest_wait.argtypes = [vp, i, p(ctypes.c_longlong)]
    lib.spec_verify_info.restype = i
    lib.spec_verify_info.argtypes = [vp, p(i), p(i), p(i), p(i), p(i)]
    lib.spec_verify_kernel_times.restype = i
    lib.spec_verify_kernel_times.argtypes = [vp, vp, i, p(i)]
    lib.spec_verify_destroy.restype = None
    lib.spec_verify_destroy.argtypes = [vp]
    lib.spec_verify_strerror.restype = ctypes.c_char_p
    lib.spec_verify_strerror.argtypes = [i]
    lib.spec_attn_init.restype = i
    lib.spec_attn_init.argtypes = [p(vp), i, i, i, i]
    lib.spec_attn_append.restype = i
    lib.spec_attn_append.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.spec_attn_read.restype = i
    lib.spec_attn_read.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.spec_attn_chunk.restype = i
    lib.spec_attn_chunk.argtypes = [vp, vp, vp, vp, i, ctypes.c_float, vp, vp, vp]
    lib.spec_attn_prompt.restype = i
    lib.spec_attn_prompt.argtypes = [vp, i, i, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]
    lib.spec_attn_get_error.restype = i
    lib.spec_attn_get_error.argtypes = [vp]
    lib.spec_attn_destroy.restype = None
    lib.spec_attn_destroy.argtypes = [vp]
    _lib = lib
    return lib
