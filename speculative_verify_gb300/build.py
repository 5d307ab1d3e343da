"""Build the sm_103a shared library in-tree with nvcc.

``build()`` compiles the translation units of ``csrc/`` (which include the
kernel headers) side by side and links them into
``speculative_verify_gb300/_build/libspecverify.so``, one ``-gencode`` for
``sm_103a``, position-independent, static CUDA runtime; and, where torch is
installed, ``csrc/layer_bind.cpp``, the Python binding of the calls between
the weight reads, against its headers (and again when torch or Python are
others).  The library needs nvcc alone.
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
BIND_SOURCE = os.path.join(CSRC, "layer_bind.cpp")
BIND_FOR = BIND_PATH + ".for"           # the torch and Python that the binding was compiled against

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")


def _lib_sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(path, sources) -> bool:
    """Whether `path` exists and none of the sources is newer."""
    return os.path.exists(path) and all(os.path.getmtime(s) <= os.path.getmtime(path) for s in sources)


def lib_up_to_date() -> bool:
    return _newer(LIB_PATH, _lib_sources())


def _bind_for(torch_root) -> str:
    """The torch (its version file) and the Python (its ABI) that a binding built now belongs to."""
    with open(os.path.join(torch_root, "version.py")) as f:
        return "%s %s\n%s" % (sysconfig.get_config_var("SOABI"), torch_root, f.read())


def bind_up_to_date(torch_root) -> bool:
    if not _newer(BIND_PATH, [BIND_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h"))]) or not os.path.exists(BIND_FOR):
        return False
    with open(BIND_FOR) as f:
        return f.read() == _bind_for(torch_root)


def _torch_root():
    """The installed torch's folder, or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else None


def _torch_paths(root):
    """(include directories, library directory) of that torch, CUDA and Python."""
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
            raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + out)
        if verbose:
            print(out)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is older than its sources -- the library, and the binding
    where torch is installed; return the library's path."""
    torch_root = _torch_root()
    lib, bind = force or not lib_up_to_date(), torch_root is not None and (force or not bind_up_to_date(torch_root))
    if not lib and not bind:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tag = ".%d.tmp" % os.getpid()
    compile_cmds, objs = [], []
    if lib:
        nvcc, flags = _nvcc(), [*ARCH_FLAGS, *NVCC_FLAGS, "-I" + INCLUDE] + (["-Xptxas=-v"] if verbose else [])
        units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
        objs = [os.path.join(BUILD_DIR, os.path.basename(u) + tag + ".o") for u in units]
        compile_cmds += [[nvcc, *flags, "-c", "-o", o, u] for u, o in zip(units, objs)]
    bind_obj = os.path.join(BUILD_DIR, "layer_bind" + tag + ".o")
    if bind:
        cxx, (torch_inc, torch_lib) = shutil.which("g++") or "g++", _torch_paths(torch_root)
        compile_cmds += [[cxx, "-std=c++17", "-O2", "-fPIC", "-Wall", "-I" + INCLUDE, *("-isystem" + d for d in torch_inc),
                          "-c", "-o", bind_obj, BIND_SOURCE]]
    try:
        _run(compile_cmds, verbose)
        if lib:
            tmp = LIB_PATH + tag
            _run([[nvcc, *ARCH_FLAGS, "-shared", "-Xlinker", "-soname=libspecverify.so", "-o", tmp, *objs]], verbose)
            os.replace(tmp, LIB_PATH)
        if bind:
            # torch's libraries are in the process before the binding is
            tmp = BIND_PATH + tag
            _run([[cxx, "-shared", "-o", tmp, bind_obj, LIB_PATH, "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu",
                   "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]],
                 verbose)
            os.replace(tmp, BIND_PATH)
            with open(tmp, "w") as f:
                f.write(_bind_for(torch_root))
            os.replace(tmp, BIND_FOR)
    finally:
        for o in [*objs, bind_obj]:
            if os.path.exists(o):
                os.remove(o)
    return LIB_PATH
