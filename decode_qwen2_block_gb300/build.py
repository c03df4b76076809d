"""Builds libblk.so in-tree with nvcc for sm_103a (GB300).

Each .cu file compiles to an object in parallel, then one shared library is
linked; beside it the Python module of csrc/binding.cpp, against torch's headers,
which calls the library that the package has loaded.  No CMake, no torch extension machinery.
"""
from __future__ import annotations

import glob
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
    files += [BINDING, os.path.abspath(__file__)]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(NATIVE):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    return all(os.path.getmtime(f) <= t for f in _deps())


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(what)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        if src == BINDING:
            inc = os.path.join(torch_dir, "include")
            _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", inc, "-I",
                  os.path.join(inc, "torch", "csrc", "api", "include"), "-I",
                  sysconfig.get_paths()["include"], "-I", os.path.join(CUDA, "include"), "-c", src,
                  "-o", obj], "g++ failed on binding.cpp", verbose)
        else:
            _run([NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj],
                 f"nvcc failed on {os.path.basename(src)}", verbose)
        return obj

    files = sources() + [BINDING]
    with ThreadPoolExecutor(max(1, min(len(files), os.cpu_count() or 1))) as ex:
        *objs, binding = ex.map(compile_one, files)
    tmp = LIB + f".tmp{os.getpid()}"
    _run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], "link of libblk.so failed")
    os.replace(tmp, LIB)
    tmp = NATIVE + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, binding, "-L", os.path.join(torch_dir, "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], "link of _native.so failed")
    os.replace(tmp, NATIVE)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
