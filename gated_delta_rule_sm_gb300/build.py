"""Build the KDA CUDA library (``libkda_gb300.so``) in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel to an object file; one nvcc call
links them into a shared library next to this file.  It exposes a plain C ABI
(``include/kda.h``) and knows nothing of torch.  The serving calls' binding
(``_ops.so``, from ``csrc/torch_ops.cpp``) is compiled beside it with the host
compiler against the installed torch, and links to it; with another torch it
is built again, and where it does not compile the library is linked all the same.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libkda_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
OPS_SRC = os.path.join(CSRC, "torch_ops.cpp")
OPS_PATH = os.path.join(PKG, "_ops.so")
OPS_TORCH = os.path.join(BUILD_DIR, "torch_ops.torch")     # the torch that _ops.so was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the KDA CUDA library cannot be built")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + [OPS_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(OPS_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(OPS_PATH))
    return all(os.path.getmtime(f) <= t for f in _deps()) and _bound_torch() == _this_torch()


def _this_torch() -> str:
    import torch
    return f"{torch.__version__} {os.path.dirname(torch.__file__)}"


def _bound_torch() -> str:
    try:
        with open(OPS_TORCH) as f:
            return f.read()
    except OSError:
        return ""


def _compile_ops() -> str:
    import sysconfig

    import torch
    top = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    includes = [INCLUDE, top, os.path.join(top, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda]
    obj = os.path.join(BUILD_DIR, "torch_ops.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f for i in includes for f in ("-isystem" if i != INCLUDE else "-I", i)], "-c", OPS_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(OPS_SRC)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ops(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = OPS_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", obj, "-o", tmp, "-L", PKG, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {os.path.basename(OPS_PATH)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS_PATH)
    with open(OPS_TORCH, "w") as f:
        f.write(_this_torch())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        ops = ex.submit(_compile_ops)
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_ops(ops.result())      # (the library is there whatever becomes of the binding)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
