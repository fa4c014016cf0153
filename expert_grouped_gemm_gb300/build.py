"""Build libmoe_gb300.so in-tree with nvcc for sm_103a.

Each .cu file under csrc/ is compiled in parallel to an object in _build/,
then all objects are linked into expert_grouped_gemm_gb300/libmoe_gb300.so
(CUDA runtime linked statically; the CUDA driver's tensor-map encoder is looked up
at run time, so no libcuda link is needed). csrc/bind.cpp, the Python module that checks
tensors and calls the library, becomes _bind.so (g++, against PyTorch's headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
BIND_STAMP = os.path.join(BUILD, "bind.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_gb300.so")
    return path


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return _sources() + [BIND_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + [
        os.path.join(PKG, "..", "include", "moe.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    return all(os.path.getmtime(d) <= t for d in _deps()) and _stamp() == bind_target()


def bind_target() -> str:
    """What _bind.so is built against: the module reads PyTorch's own structures."""
    import torch

    return f"torch {torch.__version__} python {sys.version_info[0]}.{sys.version_info[1]}"


def _stamp() -> str | None:
    try:
        with open(BIND_STAMP) as f:
            return f.read()
    except OSError:
        return None


def _compile_bind() -> None:
    import torch

    target = bind_target()
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(home, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = BIND + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DMOE_BUILT_FOR="{target}"',
           *(f"-I{d}" for d in inc), BIND_SRC, "-o", tmp, "-L" + os.path.join(home, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(BIND_STAMP, "w") as f:
        f.write(target)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(compile_one, _sources()))
        tmp = LIB + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
        bind.result()  # after the link: the experts' calls need the library alone
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
