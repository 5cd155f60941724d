"""Builds libmoe_decode.so (the CUDA kernels + the C ABI) in-tree with nvcc, and
the Python module _host.so (argument marshalling on torch tensors) with g++.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into one shared library with the CUDA runtime linked statically (the library
loads without a GPU; the driver is reached through the runtime at first use).
_host.so is built against the torch that is installed, again when that changes,
and gets the library's entry points by address. The library needs no torch: it is
linked whatever becomes of _host.so, which is left out where there is no torch.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_decode.so")
HOST = os.path.join(HERE, "_host.so")
HOST_KEY = os.path.join(BUILD, "host.key")  # the torch and the Python that _host.so was built for
SOURCES = ["api.cu", "seam.cu", "router.cu", "scales.cu", "expert.cu", "combine.cu",
           "route_static.cu", "attn_seam.cu", "add_norm.cu", "norm_add_norm.cu", "rope.cu", "kv_append.cu",
           "linear_x4.cu", "attn_x8.cu",
           "attn_x8_d64.cu", "attn_x8_d128.cu", "attn_x8_d256.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    return obj


def _link(objs: list[str]) -> None:
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def _host_key() -> str | None:
    """What _host.so is built against (None: no torch)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        return f"{sys.version}\n{spec.origin}\n{f.read()}"


def _build_host() -> None:
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = HOST + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{root}/include",
           f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
           os.path.join(CSRC, "host.cpp"), "-o", tmp, f"-L{root}/lib", "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on host.cpp:\n{r.stderr}")
    os.replace(tmp, HOST)
    with open(HOST_KEY, "w") as f:
        f.write(_host_key())


def _stale(built: str) -> bool:
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "moe_decode.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def _host_stale() -> bool:
    key = _host_key()
    if key is None:
        return False
    if _stale(HOST) or not os.path.exists(HOST_KEY):
        return True
    with open(HOST_KEY) as f:
        return f.read() != key


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile (if sources changed) and return the path of libmoe_decode.so."""
    lib, host = force or _stale(LIB), _host_key() is not None and (force or _host_stale())
    if not lib and not host:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host_done = ex.submit(_build_host) if host else None
        if lib:
            _link(list(ex.map(lambda s: _compile(s, extra), SOURCES)))
        if host_done:
            host_done.result()
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
