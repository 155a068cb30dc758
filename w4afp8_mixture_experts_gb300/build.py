"""Builds libw4a8moe.so (the CUDA library) in-tree with nvcc for sm_103a, and the Python extension beside it.

Translation units are compiled in parallel and linked with the static CUDA
runtime; the results land in w4afp8_mixture_experts_gb300/_lib/.  The extension
(w4a8_torch_ops) marshals the tensors of the operators around the routed experts;
it links to the library and holds no device code.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libw4a8moe.so")
EXT = os.path.join(LIBDIR, "w4a8_torch_ops.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "-diag-suppress", "177"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest(paths) -> float:
    return max(os.path.getmtime(p) for p in paths)


def _compile(nvcc, src, obj, deps, extra):
    if os.path.exists(obj) and os.path.getmtime(obj) >= _newest([src] + deps):
        return obj
    cmd = [nvcc] + FLAGS + extra + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_shared(srcs, out, deps, extra=(), jobs=None) -> str:
    nvcc = nvcc_path()
    os.makedirs(os.path.dirname(out), exist_ok=True)
    objs = [os.path.join(os.path.dirname(out), os.path.basename(s)[:-3] + ".o") for s in srcs]
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, os.cpu_count() or 4)) as ex:
        list(ex.map(lambda so: _compile(nvcc, so[0], so[1], deps, list(extra)), zip(srcs, objs)))
    if not (os.path.exists(out) and os.path.getmtime(out) >= _newest(objs)):
        cmd = [nvcc] + ARCH + ["-shared", "-o", out] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return out


def _torch_paths():
    """(root of the installed torch, its C++ ABI flag, its version)."""
    import torch
    return os.path.dirname(torch.__file__), int(torch._C._GLIBCXX_USE_CXX11_ABI), torch.__version__


def _torch_ops_headers() -> bool:
    """Whether the headers that the Python extension needs are installed (the CUDA library needs none of them)."""
    root = os.path.join(_torch_paths()[0], "include", "torch", "csrc")
    return (os.path.exists(os.path.join(root, "autograd", "python_variable.h"))
            and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")))


def _run_if_stale(cmd, out, deps, stamp) -> str:
    """Runs cmd to make `out`, unless it is there, newer than deps, and made by this command with this stamp (which
    stands for what cmd does not name: the versions of torch and Python)."""
    key, told = "\n".join(cmd + [stamp]), out + ".cmd"
    if os.path.exists(out) and os.path.exists(told) and os.path.getmtime(out) >= _newest(deps):
        with open(told) as f:
            if f.read() == key:
                return out
    os.makedirs(LIBDIR, exist_ok=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {out}:\n{r.stdout}\n{r.stderr}")
    with open(told, "w") as f:
        f.write(key)
    return out


def _stamp() -> str:
    return f"torch {_torch_paths()[2]}, python {sys.version}"


def _compile_torch_ops() -> str:
    """The object of the Python extension (host code only; the toolkit's headers come from nvcc's own root)."""
    src, obj = os.path.join(CSRC, "torch_ops.cpp"), os.path.join(LIBDIR, "torch_ops.o")
    root, abi, _ = _torch_paths()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"), "-isystem",
           os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem", cuda, "-c", src, "-o", obj]
    return _run_if_stale(cmd, obj, [src] + glob.glob(os.path.join(ROOT, "include", "*.h")), _stamp())


def _link_torch_ops(obj: str) -> str:
    lib = os.path.join(_torch_paths()[0], "lib")
    cmd = ["g++", "-shared", "-o", EXT, obj, "-L" + LIBDIR, "-lw4a8moe", "-L" + lib, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return _run_if_stale(cmd, EXT, [obj, LIB], _stamp())


def build() -> str:
    """The CUDA library, which needs nvcc alone, and the Python extension beside it.  Where torch's or Python's headers are
    not installed the extension is left out with a warning: the C ABI and the calls that ctypes makes need none, and the
    calls that it makes raise."""
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    if not _torch_ops_headers():
        warnings.warn("torch's or Python's headers are missing: block_norm, dense_linear and moe_route_grouped_topk are "
                      "built for the C ABI only, not for Python")
        for stale in (EXT, EXT + ".cmd"):
            if os.path.exists(stale):
                os.remove(stale)
        return build_shared(srcs, LIB, deps)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside nvcc's own jobs
        obj = ex.submit(_compile_torch_ops)
        lib = build_shared(srcs, LIB, deps)
        _link_torch_ops(obj.result())
    return lib


if __name__ == "__main__":
    print(build())
