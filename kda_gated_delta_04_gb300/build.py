"""Build libkda.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit is compiled in its own nvcc process (in parallel),
then linked into ``kda_gated_delta_04_gb300/libkda.so`` against the shared CUDA
runtime, so the library shares the process's runtime with PyTorch.

Beside it goes ``_latent_args.so`` (g++, against this interpreter's and the
installed torch's headers): the latent calls' arguments from tensors to the C
entry points without ctypes.  It is an option: where what it needs is missing, or
it cannot be compiled or linked, it is left out with a message, and kda.py passes
the same arguments through ctypes.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libkda.so")
ARGS_SRC = os.path.join(PKG, "native", "latent_args.cpp")
ARGS_PATH = os.path.join(PKG, "_latent_args.so")
HEADER = os.path.join(ROOT, "include", "kda.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA 13 toolkit required to build libkda)")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB_PATH, _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [HEADER, os.path.abspath(__file__)])


def _torch_version():
    import importlib.metadata
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _args_note():
    """Where it is kept what _latent_args.so was built for, or why it was left out."""
    return os.path.join(BUILD_DIR, "latent_args.txt")


def _args_for() -> str:
    return f"torch {_torch_version()}, {sys.implementation.cache_tag}, {platform.machine()}"


def _args_left_out():
    """Why the module was left out for this torch and interpreter, "" where it is there; None: it is to be built."""
    if not _newer(_args_note(), [ARGS_SRC, HEADER, os.path.abspath(__file__)]):
        return None
    with open(_args_note()) as f:
        made_for, _, why = f.read().partition("\n")
    if made_for != _args_for() or (not why and not os.path.exists(ARGS_PATH)):
        return None
    return why


def up_to_date() -> bool:
    return _lib_up_to_date() and _args_left_out() is not None


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and _lib_up_to_date():
        why = _args_left_out()
        if why is None:
            _link_args(*_compile_args())
        elif why:
            _say_left_out(why)
        return LIB_PATH
    nvcc = nvcc_path()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", os.path.join(ROOT, "include")]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        args_obj = ex.submit(_compile_args)
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(ARGS_PATH):  # never beside a library that it was not built for
        os.remove(ARGS_PATH)
    os.replace(tmp, LIB_PATH)
    _link_args(*args_obj.result())
    return LIB_PATH


def _compile_args():
    """The object file of latent_args.cpp and torch's library folder, or (None, why there is none)."""
    import sysconfig
    try:
        import torch
        cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    except ImportError:
        return None, "torch is not installed"
    except RuntimeError as e:
        return None, str(e)
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    py = sysconfig.get_paths()["include"]
    for need in (os.path.join(py, "Python.h"), os.path.join(inc, "torch", "csrc", "autograd", "python_variable.h"),
                 os.path.join(inc, "c10", "cuda", "CUDAStream.h"), os.path.join(libs, "libc10_cuda.so")):
        if not os.path.exists(need):
            return None, f"{need} is missing"
    obj = os.path.join(BUILD_DIR, "latent_args.o")
    why = _gxx(["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", py, "-isystem", inc,
                "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
                "-c", ARGS_SRC, "-o", obj])
    return (None, why) if why else (obj, libs)


def _gxx(args):
    """None, or why g++ with these arguments did not do it."""
    try:
        r = subprocess.run(["g++", *args], capture_output=True, text=True)
    except OSError as e:
        return f"g++: {e}"
    return None if r.returncode == 0 else f"g++ failed:\n{r.stdout}\n{r.stderr}"


def _link_args(obj, where):
    """_latent_args.so against the libkda.so that stands beside it; obj None: `where` says why not."""
    why = where
    if os.path.exists(ARGS_PATH):
        os.remove(ARGS_PATH)
    if obj is not None:
        tmp = ARGS_PATH + f".{os.getpid()}.tmp"
        why = _gxx(["-shared", "-o", tmp, obj, "-L", os.path.dirname(LIB_PATH), "-l:libkda.so", "-Wl,-rpath,$ORIGIN",
                    "-L", where, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
        if why is None:
            os.replace(tmp, ARGS_PATH)
    with open(_args_note(), "w") as f:
        f.write(f"{_args_for()}\n{why or ''}")
    if why:
        _say_left_out(why)


def _say_left_out(why):
    print(f"_latent_args left out ({why}): the latent calls go through ctypes", file=sys.stderr)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
