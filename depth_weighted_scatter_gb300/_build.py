"""Builds libbevpool.so in-tree with nvcc for sm_103a, and the native module
_token_ops of the tensor helpers.

Each .cu file under csrc/ is compiled in parallel to an object, then linked
into depth_weighted_scatter_gb300/libbevpool.so against the shared CUDA
runtime.  csrc/binding.cpp, compiled beside them by the host compiler against
PyTorch's headers, becomes _token_ops.so, which calls the library; where there
is no PyTorch (with CUDA) or no Python headers it is left out, and importing
`attention` raises.  Rebuilds only when a source is newer, the binding also when
it was made for another PyTorch or Python.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import json
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libbevpool.so")
BINDING = os.path.join(HERE, "_token_ops.so")
OBJDIR = os.path.join(ROOT, "_build")
BINDING_KEY = os.path.join(OBJDIR, "binding.json")     # what the binding was made for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def nvcc() -> str:
    p = os.path.join(CUDA_HOME, "bin", "nvcc")
    return p if os.path.exists(p) else (shutil.which("nvcc") or "nvcc")


def common_flags() -> list:
    extra = os.environ.get("BEVPOOL_NVCC_EXTRA", "").split()   # developer knob, e.g. -DBEVPOOL_FMA_VARIANT=0
    return ARCH + extra + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list:
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + [
        os.path.join(ROOT, "include", "bevpool.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(src: str, extra: list) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + common_flags() + extra + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _binding_deps() -> list:
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "bevpool.h"), os.path.abspath(__file__)]


def _torch_dir():
    """PyTorch's folder, found without importing it; None: there is none."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def binding_needs() -> list:
    """What the binding cannot be built without and is not here."""
    torch = _torch_dir()
    if torch is None:
        return ["PyTorch"]
    files = [os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(torch, "include", "c10", "cuda", "CUDAStream.h"), os.path.join(torch, "lib", "libc10_cuda.so"),
             os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    return [f for f in files if not os.path.exists(f)]


def _binding_key() -> dict:
    torch, version = _torch_dir(), ""
    if torch is not None and os.path.exists(os.path.join(torch, "version.py")):
        with open(os.path.join(torch, "version.py")) as f:
            version = f.read()
    return {"torch": torch, "version": version, "python": sys.version, "machine": platform.machine()}


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_KEY):
        return False
    t = os.path.getmtime(BINDING)
    with open(BINDING_KEY) as f:
        return all(os.path.getmtime(d) <= t for d in _binding_deps()) and json.load(f) == _binding_key()


def _compile_binding() -> str:
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJDIR, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", inc,
           "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(CUDA_HOME, "include"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L", HERE, "-l:libbevpool.so", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(BINDING_KEY):
        os.remove(BINDING_KEY)                 # a key is never older than its binding
    os.replace(tmp, BINDING)
    with open(BINDING_KEY, "w") as f:
        json.dump(_binding_key(), f)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every source and link libbevpool.so and _token_ops.so; returns
    the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    wanted, needs = force or not binding_up_to_date(), binding_needs()
    if wanted and needs:
        print("_token_ops is not built, attention cannot be imported: no " + ", ".join(needs), file=sys.stderr)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding) if wanted and not needs else None
        if force or not up_to_date():
            _build_library(verbose_ptxas)
        if binding is not None:
            _link_binding(binding.result())
    return LIB


def _build_library(verbose_ptxas: bool) -> str:
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(16, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + [
        "-Xlinker", "-rpath," + os.path.join(CUDA_HOME, "lib64")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
