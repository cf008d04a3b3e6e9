"""Builds libstq1.so in-tree: nvcc for sm_100a (device code) and g++ (host encoder).

Run ``python -m sub_bit_sparse_b200.build`` (or call ``build()``).  The library
needs only the CUDA toolkit, neither a GPU nor torch.  The CUDA runtime is
linked statically so the library does not depend on the runtime version torch
ships.

``build(debug=True)`` (``--debug``) builds libstq1_debug.so, the same sources
compiled with STQ1_DEBUG: its kernels bounds-check the indices they read
and record STQ1_DEV_BOUNDS instead of accessing out of range.  Importing the
package with STQ1_DEBUG=1 in the environment loads that library.

Where torch is installed, ``build()`` goes on to ``build_binding()``: it compiles
binding/dense_calls.cpp, the package's argument marshalling of the 8-bit and
gated calls, against that torch, and again when torch or Python have changed.
"""

from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libstq1.so")
LIB_DEBUG = os.path.join(HERE, "libstq1_debug.so")
BINDING_SRC = os.path.join(HERE, "binding", "dense_calls.cpp")
BINDING = os.path.join(HERE, "_dense_calls.so")
BINDING_FOR = os.path.join(BUILD, "dense_calls.txt")     # what the extension was compiled against
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the STQ1_0 library needs the CUDA toolkit to build")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"build step failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout, res.stderr, sep="\n")
    return res


def _sources():
    cu = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))
    cpp = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cpp"))
    hdr = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    hdr.append(os.path.join(INCLUDE, "stq1.h"))
    return cu, cpp, hdr


def up_to_date(debug: bool = False) -> bool:
    lib = LIB_DEBUG if debug else LIB
    if not os.path.exists(lib):
        return False
    cu, cpp, hdr = _sources()
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in cu + cpp + hdr + [__file__])


def _torch_version() -> str | None:
    """Version of the installed torch, found without importing it; None without torch or its CUDA libraries."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin or not os.path.exists(
            os.path.join(os.path.dirname(spec.origin), "lib", "libc10_cuda.so")):
        return None
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        return torch.__version__


def _binding_key() -> str:
    return f"torch {_torch_version()}, python {sys.version_info[0]}.{sys.version_info[1]} {sysconfig.get_config_var('SOABI')}"


def build_binding(verbose: bool = False, force: bool = False) -> str:
    """Compile the CPython extension _dense_calls.so (g++, torch's headers); returns its path."""
    inputs = [BINDING_SRC, os.path.join(INCLUDE, "stq1.h"), __file__]
    key = _binding_key()
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING_FOR):
        with open(BINDING_FOR) as f:
            same = f.read() == key
        if same and all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in inputs):
            return BINDING
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = BINDING + ".tmp"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-pthread",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[a for p in include_paths() for a in ("-isystem", p)], "-isystem", sysconfig.get_paths()["include"],
          "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
          *["-L" + p for p in library_paths()], "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_cuda", "-ltorch_python", "-ltorch"], verbose)
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_FOR, "w") as f:
        f.write(key)
    return BINDING


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False, debug: bool = False) -> str:
    """Compile every source under csrc/ into libstq1.so (libstq1_debug.so with
    debug=True) and then, where torch is installed, the binding extension;
    returns the library's path."""
    lib = LIB_DEBUG if debug else LIB
    if force or not up_to_date(debug):
        _build_library(lib, verbose, ptxas_verbose, debug)
    if _torch_version() is not None:
        build_binding(verbose, force and not debug)
    return lib


def _build_library(lib: str, verbose: bool, ptxas_verbose: bool, debug: bool) -> None:
    nvcc = _nvcc()
    build_dir = os.path.join(BUILD, "debug") if debug else BUILD
    os.makedirs(build_dir, exist_ok=True)
    cu, cpp, _ = _sources()
    objs = []
    for src in cu:
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
               "-Xcompiler", "-fPIC", "-I", INCLUDE, "-c", src, "-o", obj]
        if debug:
            cmd.insert(1, "-DSTQ1_DEBUG")
        if ptxas_verbose:
            cmd.insert(1, "-Xptxas=-v")
        _run(cmd, verbose or ptxas_verbose)
        objs.append(obj)
    for src in cpp:
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-ffp-contract=off", "-fno-fast-math",
               "-pthread", "-I", INCLUDE, "-c", src, "-o", obj]
        _run(cmd, verbose)
        objs.append(obj)
    tmp = lib + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl"], verbose)
    os.replace(tmp, lib)


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv, ptxas_verbose="--ptxas" in sys.argv,
          debug="--debug" in sys.argv)
