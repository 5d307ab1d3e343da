"""Build the sm_103a shared library in-tree with nvcc.

``build()`` compiles the translation units of ``csrc/`` (which include the
kernel headers) side by side and links them into
``speculative_verify_gb300/_build/libspecverify.so``, one ``-gencode`` for
``sm_103a``, position-independent, static CUDA runtime; and
``csrc/layer_bind.cpp``, the Python binding of the calls between the weight
reads, against the installed torch's headers.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libspecverify.so")
BIND_PATH = os.path.join(BUILD_DIR, "_layer.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BIND_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BIND_PATH))
    return all(os.path.getmtime(s) <= t for s in _sources())


def _torch_paths():
    """(include directories, library directory) of the installed torch, CUDA and Python."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is required to build the Python binding")
    root = os.path.dirname(spec.origin)
    inc = os.path.join(root, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda], \
        os.path.join(root, "lib")


def _run(cmds, verbose: bool) -> None:
    """Run the commands side by side; raise with the output of one that failed."""
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
    outs = [p.communicate()[0] for p in procs]
    for cmd, p, out in zip(cmds, procs, outs):
        if p.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + out)
        if verbose:
            print(out)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if any source is newer than it; return its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tag = ".%d.tmp" % os.getpid()
    tmp = LIB_PATH + tag
    nvcc, flags = _nvcc(), [*ARCH_FLAGS, *NVCC_FLAGS, "-I" + INCLUDE] + (["-Xptxas=-v"] if verbose else [])
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(BUILD_DIR, os.path.basename(u) + tag + ".o") for u in units]
    bind_obj, bind_tmp = os.path.join(BUILD_DIR, "layer_bind" + tag + ".o"), BIND_PATH + tag
    torch_inc, torch_lib = _torch_paths()
    cxx = shutil.which("g++") or "g++"
    try:
        _run([[nvcc, *flags, "-c", "-o", o, u] for u, o in zip(units, objs)]
             + [[cxx, "-std=c++17", "-O2", "-fPIC", "-Wall", "-I" + INCLUDE, *("-isystem" + d for d in torch_inc), "-c",
                 "-o", bind_obj, os.path.join(CSRC, "layer_bind.cpp")]], verbose)
        _run([[nvcc, *ARCH_FLAGS, "-shared", "-Xlinker", "-soname=libspecverify.so", "-o", tmp, *objs]], verbose)
        os.replace(tmp, LIB_PATH)
        # torch's libraries are in the process before the binding is
        _run([[cxx, "-shared", "-o", bind_tmp, bind_obj, LIB_PATH, "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu",
               "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]],
             verbose)
        os.replace(bind_tmp, BIND_PATH)
    finally:
        for o in [*objs, bind_obj]:
            if os.path.exists(o):
                os.remove(o)
    return LIB_PATH
