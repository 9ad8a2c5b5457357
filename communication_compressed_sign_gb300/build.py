"""Build the lioncub CUDA library (liblioncub.so) in-tree for sm_103a.

Each .cu file under csrc/ is compiled in parallel with nvcc and the objects
are linked into one shared library with the C ABIs of include/lioncub.h,
include/lioncub_embed.h and include/lioncub_block.h.  No PyTorch headers or types are
involved: the library is plain CUDA C++ with the CUDA runtime linked statically.
Beside it a small Python module, _tensors, is compiled against the installed
torch: it reads the block operators' arguments from tensors and calls the library.

    python -m communication_compressed_sign_gb300.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblioncub.so")
OBJ_DIR = os.path.join(PKG, "_build")
# The same library with every kernel index validated in-kernel (violations set
# a status bit instead of touching memory); used by the tests as a stand-in
# for a memory checker.
CHECKED_LIB = os.path.join(PKG, "liblioncub_checked.so")

TENSORS = os.path.join(PKG, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))
TENSORS_SOURCE = os.path.join(CSRC, "tensors.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-fmad=false", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr", *ARCH]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the lioncub CUDA library cannot be built")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
             if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in ("lioncub.h", "lioncub_embed.h", "lioncub_block.h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, bounds_check: bool = False) -> str:
    lib = CHECKED_LIB if bounds_check else LIB
    obj_dir = os.path.join(OBJ_DIR, "checked") if bounds_check else OBJ_DIR
    if not force and up_to_date(lib):
        return lib
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []
    if bounds_check:
        extra.append("-DLIONCUB_BOUNDS_CHECK")

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra, f"-I{INCLUDE}", f"-I{CSRC}", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def _torch_dir() -> str | None:
    """Where torch is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def build_tensors(force: bool = False) -> str | None:
    """Compile the _tensors module; it needs torch's and Python's headers and a C++ compiler.

    Without those headers nothing else needs it (its users say that it is missing): None then.
    """
    torch, python = _torch_dir(), sysconfig.get_paths()["include"]
    if torch is None or not os.path.exists(os.path.join(python, "Python.h")):
        print(f"{'torch is not installed' if torch is None else 'there is no Python.h'}: the _tensors module is not built",
              file=sys.stderr)
        return None
    version = os.path.join(torch, "version.py")
    inputs = [TENSORS_SOURCE, version, os.path.abspath(__file__),
              *(os.path.join(INCLUDE, f) for f in ("lioncub.h", "lioncub_embed.h", "lioncub_block.h"))]
    if not force and os.path.exists(TENSORS) and all(os.path.getmtime(f) <= os.path.getmtime(TENSORS) for f in inputs):
        return TENSORS
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler: the _tensors module cannot be built")
    tmp, libs = TENSORS + f".tmp{os.getpid()}", os.path.join(torch, "lib")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f"-I{INCLUDE}", f"-I{os.path.join(torch, 'include')}",
           f"-I{os.path.join(torch, 'include', 'torch', 'csrc', 'api', 'include')}", f"-I{python}",
           TENSORS_SOURCE, "-o", tmp, f"-L{libs}", "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on {TENSORS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSORS)
    return TENSORS


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv, bounds_check="--bounds-check" in sys.argv))
    if tensors := build_tensors(force=True):
        print(tensors)
