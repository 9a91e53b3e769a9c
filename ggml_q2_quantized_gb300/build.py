"""Build libq2k.so in-tree with nvcc for sm_103a (no cmake).

Each ``csrc/*.cu`` compiles to an object in parallel; the objects link into
``_build/libq2k.so`` with the CUDA runtime linked statically, so the library
needs only the NVIDIA driver at run time.  Where PyTorch is installed, g++ builds
the module through which its tensors reach the feed-forward calls
(``csrc/q2k_torch.cpp``; one file for each PyTorch version).  ``python -m
ggml_q2_quantized_gb300.build`` does the same from the command line.
"""

from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libq2k.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3", "-lineinfo", "-std=c++17", "--fmad=true",
    "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libq2k")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, verbose_ptxas: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def torch_module_path(version: str) -> str:
    """Where the module for a PyTorch version lies."""
    return os.path.join(BUILD_DIR, f"q2k_torch-{version}.so")


def build_torch_module(force: bool = False) -> str | None:
    """Compile q2k_torch for the installed PyTorch if its sources changed; return its
    path, or None without PyTorch."""
    if importlib.util.find_spec("torch") is None:
        return None
    import torch

    src = os.path.join(CSRC, "q2k_torch.cpp")
    path = torch_module_path(torch.__version__)
    deps = [src] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(path) and all(
            os.path.getmtime(p) <= os.path.getmtime(path) for p in deps):
        return path
    os.makedirs(BUILD_DIR, exist_ok=True)
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(home, "include"),
           "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), src, "-o", tmp,
           "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if os.path.exists(path):
        os.remove(path)  # (one of other sources must not be loaded if this fails)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libq2k.so, and the module for PyTorch where that is
    installed, if any source changed; return the library's path.  The package runs
    without the module, so where it does not compile (no Python headers, say) that is
    a warning."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(build_torch_module, force)
        path = _build_library(force, verbose_ptxas)
        try:
            module.result()
        except Exception as e:  # noqa: BLE001 (whatever it is, the library is there)
            warnings.warn(f"the PyTorch module was not built; feed-forward calls go through ctypes: {e}",
                          RuntimeWarning, stacklevel=2)
    return path


def _build_library(force: bool, verbose_ptxas: bool) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    log = "".join(err for _, err in results)
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
