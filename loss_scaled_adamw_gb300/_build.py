"""Build the CUDA library (libtl_gb300.so) in-tree with nvcc for sm_103a.

The translation units (kernels, host C ABI, the allocation-free entry point, the
objectives over logits) compile in parallel, then link into one shared library with
the CUDA runtime linked statically.  The objectives' binding (_loss_bind, a CPython
module over torch's headers) is host code of its own beside it, and nothing of the
optimizer step needs it.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtl_gb300.so")
SOURCES = ["tl_kernels.cu", "tl_kernels_split.cu", "tl_api.cu", "tl_noalloc.cu", "tl_loss_kernels.cu", "tl_stats_kernels.cu",
           "tl_loss_api.cu", "tl_dropout.cu"]
HEADERS = [os.path.join(CSRC, "tl_internal.cuh"), os.path.join(CSRC, "tl_loss_internal.cuh"),
           os.path.join(CSRC, "tl_loss_device.cuh"), os.path.join(CSRC, "tl_spans.h"),
           os.path.join(ROOT, "include", "tl.h"), os.path.join(ROOT, "include", "tl_loss.h"),
           os.path.join(ROOT, "include", "tl_dropout.h")]
BIND = os.path.join(PKG, "_loss_bind.so")
BIND_SOURCE = os.path.join(CSRC, "tl_loss_bind.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-fmad=false", "-Xcompiler", "-fPIC",
                     "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library and the objectives' binding where a source or header is newer."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if force or _stale(LIB, srcs + HEADERS + [__file__]):
        _build_library(srcs, verbose)
    if force or _stale(BIND, [BIND_SOURCE, __file__] + HEADERS) or _built_key() != _binding_key():
        _build_binding(verbose)
    return LIB


def _binding_key() -> str:
    """What the binding is compiled against: a torch and a Python of some version."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"{sysconfig.get_config_var('SOABI')} torch {version}"


def _built_key() -> str:
    path = os.path.join(BUILD, "_loss_bind.key")
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _run(cmd, verbose: bool, what: str) -> None:
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + " ".join(cmd) + "\n" + r.stdout)


def _build_binding(verbose: bool) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return   # the optimizer step's binding does without torch; losses.py says what is missing
    torch = os.path.dirname(spec.origin)
    tmp = BIND + f".tmp{os.getpid()}"
    try:
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I" + sysconfig.get_path("include"),
              "-isystem", os.path.join(torch, "include"),
              "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"), BIND_SOURCE, "-o", tmp,
              "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(torch, "lib"),
              "-ltorch_python", "-ltorch_cpu", "-lc10"], verbose, "g++")
    except (OSError, RuntimeError) as e:
        # no compiler, or no headers of Python or torch: the library stands without the binding, and
        # the objectives' calls say that it is missing.  An older one may pass other structures.
        if os.path.exists(BIND):
            os.remove(BIND)
        warnings.warn(f"the objectives' binding was not built; the optimizer step does not need it: {e}", RuntimeWarning)
        return
    os.replace(tmp, BIND)
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, "_loss_bind.key"), "w") as f:
        f.write(_binding_key())


def _build_library(srcs, verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    objs, procs = [], []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + out)
        if verbose and out:
            print(out)
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], verbose, "link")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
