"""Build libmla.so (the CUDA library behind include/mla.h) for sm_103a with nvcc.

Each translation unit compiles in its own nvcc process (in parallel); the objects link into
``mla_latent_cache_attention_gb300/_build/libmla.so`` against the shared CUDA runtime.  Beside it,
``mla_marshal`` is the C marshalling of the selector's Python calls (linked to libmla.so), named with the
interpreter's ABI: another one builds its own.  Where it cannot be built (no Python headers) the library stands
without it, and those calls take their Python form.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmla.so")
MARSHAL = os.path.join(BUILD, "mla_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["mla_api.cu", "mla_small_kernels.cu", "mla_attn_bf16.cu", "mla_attn_fp8.cu", "mla_attn_ds.cu",
           "mla_noalloc.cu", "mla_paged_tma_bf16.cu", "mla_paged_tma_fp8.cu", "mla_ds.cu", "mla_fp4.cu", "mla_head_bmm.cu",
           "mla_index.cu", "mla_index_scores.cu", "mla_index_api.cu", "mla_rope.cu", "mla_plan.cu", "mla_step_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "mla.h"), __file__]
    return [f for f in files if os.path.isfile(f)]


def _newer_than_inputs(path) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in _inputs())


def up_to_date() -> bool:
    return _newer_than_inputs(LIB) and _newer_than_inputs(MARSHAL)


def build_marshal() -> bool:
    """Build the C marshalling for this interpreter; where that fails, warn and leave none (not an old one either)."""
    include = sysconfig.get_paths()["include"]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    if os.path.exists(os.path.join(include, "Python.h")):
        cmd = [nvcc(), "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-I", include, "-I", INCLUDE, "-shared", "-cudart", "shared",
               os.path.join(CSRC, "mla_marshal.cpp"), "-o", tmp, "-L", os.path.dirname(LIB), "-lmla", "-Xlinker", "-rpath=$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = "" if r.returncode == 0 else r.stdout + r.stderr
    else:
        why = f"no Python.h in {include}"
    if not why:
        os.replace(tmp, MARSHAL)
        return True
    for f in (tmp, MARSHAL):
        if os.path.exists(f):
            os.remove(f)
    warnings.warn(f"the selector's calls take their Python form, mla_marshal could not be built: {why}")
    return False


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    if not force and _newer_than_inputs(LIB):
        build_marshal()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nv = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nv, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nv, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_marshal()
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(force=True, verbose=v, extra=(["-Xptxas", "-v"] if v else [])))
