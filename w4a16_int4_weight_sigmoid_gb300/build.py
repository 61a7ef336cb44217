"""Build libchord_moe.so (sm_103a) in-tree with nvcc, and its Python extension.

Each .cu under csrc/ is compiled in parallel to an object under _build/,
then linked into w4a16_int4_weight_sigmoid_gb300/libchord_moe.so; meanwhile
csrc_py/binding.cpp is compiled against the installed torch and then linked
to the library as w4a16_int4_weight_sigmoid_gb300/_chord.so.  A source or
header newer than what is built from it triggers a rebuild, and for the
extension another torch or Python than it was compiled against.  Where the
extension cannot be built (no C++ compiler, Python.h or torch headers) the
library is there all the same, with a warning; calls that need the extension
raise.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libchord_moe.so")
EXT_SRC = os.path.join(HERE, "csrc_py", "binding.cpp")
EXT_PATH = os.path.join(HERE, "_chord.so")
EXT_STAMP = os.path.join(BUILD_DIR, "binding.torch")   # what the extension was compiled against
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _against() -> str:
    try:
        import torch
    except ImportError:
        return ""
    return f"torch {torch.__version__}, Python {sys.version}"


def _lib_up_to_date() -> bool:
    return _newer(LIB_PATH, _sources() + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def _ext_up_to_date() -> bool:
    if not _newer(EXT_PATH, [EXT_SRC] + _headers()) or not os.path.exists(EXT_STAMP):
        return False
    with open(EXT_STAMP) as f:
        return f.read() == _against()


def up_to_date() -> bool:
    return _lib_up_to_date() and _ext_up_to_date()


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
    with open(EXT_STAMP, "w") as f:
        f.write(_against())


def _build_lib(extra_flags) -> None:
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), srcs))
    tmp = LIB_PATH + ".tmp"
    _run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB_PATH)


def _build_ext(compiled) -> None:
    """Links what `compiled` (a future of _compile_ext) gives.  A failure leaves no extension
    behind: one of other headers or another torch must not be loaded."""
    try:
        _link_ext(compiled.result())
    except (RuntimeError, OSError, ImportError) as e:
        if os.path.exists(EXT_PATH):
            os.remove(EXT_PATH)
        warnings.warn(f"the library is built, its Python extension is not: {e}", RuntimeWarning)


def build(force: bool = False, extra_flags=(), verbose: bool = False) -> str:
    """Compile and link what is out of date; returns the library's path."""
    force = force or bool(extra_flags)
    lib, ext = force or not _lib_up_to_date(), force or not _ext_up_to_date()
    if not lib and not ext:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as pool:
        compiled = pool.submit(_compile_ext) if ext else None
        if lib:
            _build_lib(extra_flags)
    if ext:
        _build_ext(compiled)
    if verbose:
        print("built", LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose=True)
