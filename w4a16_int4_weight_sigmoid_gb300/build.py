"""Build libchord_moe.so (sm_103a) in-tree with nvcc, and its Python extension.

Each .cu under csrc/ is compiled in parallel to an object under _build/,
then linked into w4a16_int4_weight_sigmoid_gb300/libchord_moe.so; meanwhile
csrc_py/binding.cpp is compiled against the installed torch and then linked
to the library as w4a16_int4_weight_sigmoid_gb300/_chord.so.  A source or
header newer than the library triggers a rebuild.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libchord_moe.so")
EXT_SRC = os.path.join(HERE, "csrc_py", "binding.cpp")
EXT_PATH = os.path.join(HERE, "_chord.so")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [EXT_SRC, os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(EXT_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(EXT_PATH))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_ext() -> str:
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD_DIR, "binding.o")
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-w", "-I", INCLUDE, "-I", root,
          "-I", os.path.join(root, "torch", "csrc", "api", "include"),
          "-I", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
          "-I", sysconfig.get_paths()["include"],
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", EXT_SRC, "-o", obj],
         f"compiling {EXT_SRC}")
    return obj


def _link_ext(obj: str) -> None:
    import torch
    tmp = EXT_PATH + ".tmp"
    _run([CXX, "-shared", "-o", tmp, obj, "-L", HERE, "-lchord_moe", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python"], f"linking {EXT_PATH}")
    os.replace(tmp, EXT_PATH)


def build(force: bool = False, extra_flags=(), verbose: bool = False) -> str:
    """Compile and link the library; returns its path."""
    if not force and not extra_flags and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), srcs))
        ext_obj = ext.result()
    tmp = LIB_PATH + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_ext(ext_obj)
    if verbose:
        print("built", LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose=True)
