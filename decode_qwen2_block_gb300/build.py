"""Builds libblk.so in-tree with nvcc for sm_103a (GB300).

Each .cu file compiles to an object in parallel, then one shared library is
linked; beside it the Python module of csrc/binding.cpp, against torch's headers,
which calls the library that the package has loaded.  No CMake, no torch extension machinery.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libblk.so")
NATIVE = os.path.join(HERE, "_native.so")
NATIVE_TAG = os.path.join(BUILD, "native.tag")
BINDING = os.path.join(CSRC, "binding.cpp")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    files = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files.append(os.path.join(os.path.dirname(HERE), "include", "blk.h"))
    files.append(os.path.abspath(__file__))
    return files


def _torch_dir():
    """Where torch is, or None without it."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _native_tag() -> str:
    """What the module is built against: it serves this Python and this torch alone."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return f"{sysconfig.get_config_var('SOABI')} torch {version} in {_torch_dir()}"


def _newer(target: str, files) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def _native_up_to_date() -> bool:
    if not _newer(NATIVE, [BINDING, *_deps()]) or not os.path.exists(NATIVE_TAG):
        return False
    with open(NATIVE_TAG) as f:
        return f.read() == _native_tag()


def up_to_date() -> bool:
    """The library, and the module where there is a torch to build it against."""
    return _newer(LIB, _deps()) and (_torch_dir() is None or _native_up_to_date())


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(what)


def _compile(src, verbose, extra):
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
    _run([NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj],
         f"nvcc failed on {os.path.basename(src)}", verbose)
    return obj


def _build_native(torch_dir, verbose):
    inc = os.path.join(torch_dir, "include")
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", inc, "-I",
          os.path.join(inc, "torch", "csrc", "api", "include"), "-I",
          sysconfig.get_paths()["include"], "-I", os.path.join(CUDA, "include"), "-c", BINDING,
          "-o", obj], "g++ failed on binding.cpp", verbose)
    tmp = NATIVE + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(torch_dir, "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], "link of _native.so failed")
    os.replace(tmp, NATIVE)
    with open(NATIVE_TAG, "w") as f:
        f.write(_native_tag())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The library first, for which nothing of Python is needed; what the module lacks is
    raised behind it.  Without torch there is no module (the C ABI and the calls that go
    through ctypes are there)."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    torch_dir = _torch_dir()
    with ThreadPoolExecutor(max(1, min(len(sources()) + 1, os.cpu_count() or 1))) as ex:
        native = None
        if torch_dir is None:
            sys.stderr.write("no torch: _native.so, the module of the paged calls, is left out\n")
        elif force or not _native_up_to_date():
            native = ex.submit(_build_native, torch_dir, verbose)
        if force or not _newer(LIB, _deps()):
            objs = list(ex.map(lambda src: _compile(src, verbose, extra), sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], "link of libblk.so failed")
            os.replace(tmp, LIB)
        if native is not None:
            native.result()
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
