"""In-tree build of libbastion.so (nvcc, sm_103a only).

Each CUDA translation unit compiles in parallel; the shared library links the
CUDA runtime statically so it loads without a separate libcudart.  Beside it
gcc compiles a small CPython extension (csrc/marshal.c), the paged cache's short
way from Python into the library; where that cannot be built, the library stands
without it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libbastion.so")
# csrc/marshal.c, a CPython extension; it is built against one interpreter's C API, which its name says
MARSHAL = os.path.join(BUILD, "bastion_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.cu", "topk_marginals.cu", "build_tree.cu", "verify_greedy.cu", "tree_attention.cu",
           "verify_noalloc.cu", "verify_sample.cu", "calibrate.cu",
           "build_tree_mixture.cu", "lm_head_topk.cu",
           "api_cache.cu", "paged_append.cu", "paged_attention.cu", "paged_evict.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in ("bastion.h", "bastion_cache.h")]
    return files


def _newer(path, inputs) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def marshal_up_to_date() -> bool:
    files = [os.path.join(CSRC, "marshal.c")] + [os.path.join(INCLUDE, f) for f in ("bastion.h", "bastion_cache.h")]
    return _newer(MARSHAL, [f for f in files if os.path.exists(f)])  # a built tree may come without its sources


def build_marshal() -> None:
    """The extension, or a warning that says why there is none."""
    tmp = MARSHAL + f".tmp{os.getpid()}"
    try:
        r = subprocess.run(["gcc", "-O2", "-std=gnu11", "-fPIC", "-shared", "-Wall", "-I", INCLUDE, "-I",
                            sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.c"), "-o", tmp],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise OSError(r.stderr[-2000:])
        os.replace(tmp, MARSHAL)
    except OSError as e:
        warnings.warn(f"csrc/marshal.c could not be built (the paged cache's calls take the way through ctypes): {e}")


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        _build_library()
    if force or not marshal_up_to_date():
        build_marshal()
    if verbose:
        print(f"built {LIB}")
    return LIB


def _build_library() -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
               "-Xptxas", "-v", "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        with open(obj + ".log", "w") as f:
            f.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force=True, verbose=True)
