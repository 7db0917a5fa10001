"""Build the CUDA library ``libmha.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` file is compiled by nvcc to an object in parallel, then the
objects are linked into ``transformer_head_scaled_fwd_gb300/libmha.so``
(static CUDA runtime, no libcuda link: the tensor-map encoder is fetched from
the driver at run time). Rebuilds only when a source or header is newer than
the library.

``build(debug=True)`` builds ``libmha_debug.so`` instead: the same sources with
MHA_DEVICE_CHECKS defined, so the kernels check their block and tile indices at
entry and record a status code (mha_check_device_status) instead of touching
memory when one falls outside the problem.

``build()`` also compiles ``csrc/front.cpp`` (the host compiler, torch's headers)
into ``_front.so``, through which the Python binding makes the serving calls.
Where it does not compile (no headers of torch or Python, a torch without CUDA) it is left
out with a message, and the binding uses ctypes.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmha.so")
LIB_DEBUG = os.path.join(PKG, "libmha_debug.so")
FRONT = os.path.join(PKG, "_front.so")
FRONT_SRC = os.path.join(CSRC, "front.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libmha.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(CSRC, "*.inc")) + [os.path.join(ROOT, "include", "mha.h"), __file__])


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps())


def build_front(force: bool = False):
    """Compile _front.so for this interpreter and the installed torch; None where that cannot be done."""
    spec = importlib.util.find_spec("torch")
    torch = os.path.dirname(spec.origin) if spec is not None and spec.origin else None
    python = sysconfig.get_paths()["include"]
    gxx = shutil.which("g++")
    if (torch is None or gxx is None or not os.path.exists(os.path.join(python, "Python.h"))
            or not os.path.exists(os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h"))):
        print("_front.so is not built: g++ or the headers of Python or torch are missing", file=sys.stderr)
        return None
    stamp = os.path.join(BUILD, "front.stamp")
    made_for = f"{sys.version}\n{importlib.metadata.version('torch')}\n{torch}\n"
    deps = [FRONT_SRC, os.path.join(ROOT, "include", "mha.h"), __file__]
    if not force and os.path.exists(FRONT) and os.path.exists(stamp) and open(stamp).read() == made_for \
            and all(os.path.getmtime(p) <= os.path.getmtime(FRONT) for p in deps):
        return FRONT
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    include = [python, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"), cuda]
    libs = os.path.join(torch, "lib")
    tmp = FRONT + f".tmp{os.getpid()}"
    r = subprocess.run([gxx, "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{p}" for p in include), FRONT_SRC, "-o", tmp,
                        f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{libs}"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(FRONT):   # of other sources, or another torch
            os.remove(FRONT)
        print(f"_front.so is not built: g++ failed on {os.path.basename(FRONT_SRC)}:\n{r.stderr}", file=sys.stderr)
        return None
    os.replace(tmp, FRONT)
    with open(stamp, "w") as f:
        f.write(made_for)
    return FRONT


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    if not debug:
        with cf.ThreadPoolExecutor(max_workers=1) as ex:   # beside nvcc
            front = ex.submit(build_front, force)
            lib = _build_library(lib, force, verbose, extra_flags, debug)
            front.result()
        return lib
    return _build_library(lib, force, verbose, extra_flags, debug)


def _build_library(lib, force, verbose, extra_flags, debug) -> str:
    if not force and not needs_build(lib):
        return lib
    out_dir = BUILD + ("_debug" if debug else "")
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    flags = list(extra_flags) + (["-DMHA_DEVICE_CHECKS"] if debug else [])
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", os.path.join(ROOT, "include"), *flags]

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src) + ".o")
        cmd = common + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    v = "-v" in sys.argv
    flags = ["-Xptxas", "-v"] if v else []
    print(build(force=True, verbose=v, extra_flags=flags))
