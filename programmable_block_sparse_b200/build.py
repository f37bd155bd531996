"""Build the CUDA library ``libflexattn_b200.so`` in-tree with nvcc (sm_100a).

Every ``csrc/*.cu`` is compiled to an object under ``_build/`` at the repo
root and linked into ``programmable_block_sparse_b200/libflexattn_b200.so``.
Objects are rebuilt when their source, or any header under ``csrc/`` or
``include/``, is newer.  ``csrc/binding.cpp`` is compiled with g++ against
torch's headers into ``_binding.so`` beside the library, again whenever torch or
the interpreter is another one.  Where that cannot be done (no headers), the
library is built all the same, and only the calls that go through the binding
raise.  Usage: ``python -m programmable_block_sparse_b200.build``.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libflexattn_b200.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "binding.stamp")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-I" + INCLUDE, "-I" + CSRC,
]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build the library")


def _newest_header():
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(nvcc, src, obj, verbose):
    cmd = [nvcc] + NVCC_FLAGS + ["-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return r.stderr if verbose else ""


def _binding_key():
    """What the binding's ABI depends on beside its sources: torch and the interpreter."""
    from importlib.metadata import PackageNotFoundError, version
    try:
        torch_version = version("torch")
    except PackageNotFoundError:
        torch_version = "none"
    return f"torch {torch_version}, {sys.implementation.cache_tag}\n"


def _binding_is_current():
    """Newer than its sources, and built against this torch and interpreter."""
    newest = max(os.path.getmtime(BINDING_SRC), os.path.getmtime(os.path.join(INCLUDE, "flexattn.h")))
    if not os.path.exists(BINDING_PATH) or os.path.getmtime(BINDING_PATH) < newest or not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP) as f:
        return f.read() == _binding_key()


def _build_binding():
    """csrc/binding.cpp -> _binding.so, next to the library it calls."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-DTORCH_EXTENSION_NAME=_binding",
           "-DTORCH_API_INCLUDE_EXTENSION_H", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += ["-I" + d for d in includes] + [BINDING_SRC, "-o", tmp, "-L" + PKG_DIR, "-lflexattn_b200",
                                           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
                                           "-ltorch_cuda", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(force=False, verbose=False, jobs=None):
    """Compile and link; returns the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    todo, objs = [], []
    for src in sources:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time):
            todo.append((src, obj))
    logs = []
    if todo:
        with ThreadPoolExecutor(max_workers=jobs or min(len(todo), os.cpu_count() or 4)) as ex:
            logs = list(ex.map(lambda so: _compile(nvcc, so[0], so[1], verbose), todo))
    if todo or force or not os.path.exists(LIB_PATH):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc] + ARCH_FLAGS + ["-shared", "-o", tmp] + objs + ["-cudart", "static", "-ldl", "-lrt", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    if verbose:
        for log in logs:
            sys.stderr.write(log)
    if force or not _binding_is_current():
        for path in (BINDING_PATH, BINDING_STAMP):  # never one of another ABI
            if os.path.exists(path):
                os.remove(path)
        try:
            _build_binding()
        except (ImportError, OSError, RuntimeError) as e:
            sys.stderr.write(f"the compiled binding was not built; the calls that need it will raise: {e}\n")
        else:
            with open(BINDING_STAMP, "w") as f:
                f.write(_binding_key())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    sys.exit(0 if os.path.exists(BINDING_PATH) else 1)
