"""Build libfa.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a.

Each translation unit is compiled to an object in parallel, then linked into
``exact_attention_33_gb300/libfa.so``.  No cmake; only nvcc and the host
compiler.  Run as ``python -m exact_attention_33_gb300.build`` or through
``__graft_entry__.build()``.

``--checked`` (``build(checked=True)``) builds the same sources with
FA_DEBUG_CHECKS into ``libfa_checked.so``: every plain global load and store of
the kernels is checked against its buffer's extent, and a failing access is
skipped and reported in the status word (FA_DEV_BAD_INDEX).  The binding loads
that library when the environment sets FA_CHECKED=1.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfa.so")
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libfa_checked.so")
# the binding's short way for calls on torch tensors (csrc/torch_calls.cpp)
TORCH_CALLS = os.path.join(PKG, "_torch_calls.so")
SOURCES = ["fa_api.cu", "fa_cache_api.cu", "prefill.cu", "prefill_window.cu", "prefill_fp8cache.cu",
           "decode.cu", "decode_fp8.cu", "cache_append.cu", "backward.cu", "backward_window.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put /usr/local/cuda/bin on PATH)")


def common_flags():
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                   "-I" + os.path.join(PKG, "..", "include"), "--expt-relaxed-constexpr"]


def torch_calls_command(out):
    """g++ command for the extension module: torch's and Python's headers, no
    nvcc.  It needs no symbols of libfa.so (their addresses are bound at run
    time)."""
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    lib = os.path.join(root, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(root, "include"),
            "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(cuda, "include"),
            "-I", os.path.join(PKG, "..", "include"),
            os.path.join(CSRC, "torch_calls.cpp"), "-o", out,
            "-L", lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed:\n" + " ".join(cmd) + "\n" + r.stdout)
    if verbose and r.stdout.strip():
        print(r.stdout, flush=True)
    return r.stdout


def _newer(path, deps):
    """``path`` exists and is no older than any of ``deps``."""
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _build_torch_calls(verbose):
    """The extension module, or a warning: the binding makes its calls without it."""
    tmp = TORCH_CALLS + ".tmp"
    try:
        _run(torch_calls_command(tmp), verbose)
        os.replace(tmp, TORCH_CALLS)
    except Exception as e:
        if os.path.exists(TORCH_CALLS):  # made from older headers: not to be bound
            os.remove(TORCH_CALLS)
        warnings.warn(f"calls on torch tensors take longer without {TORCH_CALLS}: {e}",
                      RuntimeWarning)


def build(verbose: bool = False, ptxas_verbose: bool = False, force: bool = False,
          checked: bool = False) -> str:
    """Compile every CUDA source and link libfa.so (libfa_checked.so with
    ``checked``); returns the library path.  The library needs nvcc alone; the
    extension module beside it is left out with a warning where it does not
    compile."""
    nvcc = nvcc_path()
    build_dir, lib = (BUILD_CHECKED, LIB_CHECKED) if checked else (BUILD, LIB)
    defines = ["-DFA_DEBUG_CHECKS"] if checked else []
    os.makedirs(build_dir, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    inc = os.path.join(PKG, "..", "include")
    api = [os.path.join(inc, h) for h in os.listdir(inc)]
    deps = api + srcs + [os.path.join(CSRC, h) for h in os.listdir(CSRC)
                         if h.endswith((".h", ".cuh"))]
    lib_ready = not force and _newer(lib, deps)
    # (one module serves both builds)
    calls_ready = not force and _newer(TORCH_CALLS, api + [os.path.join(CSRC, "torch_calls.cpp")])

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc] + common_flags() + defines + ["-c", src, "-o", obj]
        if ptxas_verbose:
            cmd += ["-Xptxas", "-v"]
        out = _run(cmd, verbose)
        if ptxas_verbose and out:
            print(out, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        calls = None if calls_ready else ex.submit(_build_torch_calls, verbose)
        if not lib_ready:
            objs = list(ex.map(compile_one, srcs))
            tmp = lib + ".tmp"
            _run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs, verbose)
            os.replace(tmp, lib)
        if calls is not None:
            calls.result()
    return lib


if __name__ == "__main__":
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv, force="-f" in sys.argv,
                checked="--checked" in sys.argv))
