"""Build libcalibatt.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a,
and _pycalls.so (its streaming calls without ctypes) against the installed torch.

    python -m calibrated_block_sparse_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libcalibatt.so")
PYCALLS = os.path.join(HERE, "_pycalls.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def needs_build() -> bool:
    if not os.path.exists(LIB) or (not os.path.exists(PYCALLS) and pycalls_command(LIB, "") is not None):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [os.path.join(CSRC, "pycalls.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int = 4, out_path: str = None,
          defines=()) -> str:
    """Compile every csrc/*.cu and link libcalibatt.so (in-tree unless out_path)."""
    target = out_path or LIB
    if not force and not defines and out_path is None and not needs_build():
        return LIB
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                    "--expt-relaxed-constexpr"]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    flags += [f"-D{d}" for d in defines]
    pycalls = start_pycalls(cc) if out_path is None else None
    try:
        return _build(cc, flags, jobs, target, pycalls)
    finally:
        if pycalls is not None:
            pycalls[0].wait()
            if os.path.exists(pycalls[1]):
                os.remove(pycalls[1])


def _build(cc, flags, jobs, target, pycalls):
    with tempfile.TemporaryDirectory(prefix="calibatt_build_") as tmp:
        objs = []
        procs = []
        for src in sources():
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            objs.append(obj)
            procs.append(subprocess.Popen([cc, *flags, "-c", src, "-o", obj]))
            if len(procs) >= jobs:
                if procs.pop(0).wait() != 0:
                    raise RuntimeError("nvcc failed")
        for p in procs:
            if p.wait() != 0:
                raise RuntimeError("nvcc failed")
        out = target + f".tmp{os.getpid()}"
        subprocess.check_call([cc, *ARCH, "-shared", "-o", out, *objs, "-lcudart_static", "-ldl", "-lpthread",
                               "-lrt"])
        if target == LIB and os.path.exists(PYCALLS):
            # it calls the library by address: one of another build may pass other arguments
            os.remove(PYCALLS)
        os.replace(out, target)
    if pycalls is not None:
        process, made = pycalls
        if process.wait() == 0:
            os.replace(made, PYCALLS)
        else:
            warnings.warn("compiling pycalls.cpp failed: the streaming calls go through ctypes", RuntimeWarning)
    return target


def start_pycalls(cc):
    """Starts compiling csrc/pycalls.cpp: the process and the file it makes, or
    None where it cannot be made."""
    out = PYCALLS + f".tmp{os.getpid()}"
    command = pycalls_command(cc, out)
    return None if command is None else (subprocess.Popen(command), out)


def pycalls_command(cc, out):
    """The compiler's call for csrc/pycalls.cpp, or None without a C++ compiler
    or the headers of Python or torch."""
    gxx, include = shutil.which("g++") or shutil.which("c++"), sysconfig.get_paths()["include"]
    spec = importlib.util.find_spec("torch")
    if gxx is None or spec is None or not os.path.exists(os.path.join(include, "Python.h")):
        return None
    torch = spec.submodule_search_locations[0]
    if not os.path.exists(os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return None
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"__version__ = ['\"]([^'\"]+)['\"]", f.read()).group(1)
    headers = [include, INCLUDE, os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")]
    return [gxx, "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", f'-DCALIBATT_TORCH="{version}"',
            *(f"-I{x}" for x in headers), os.path.join(CSRC, "pycalls.cpp"), "-o", out,
            "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


if __name__ == "__main__":
    print(build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv))
