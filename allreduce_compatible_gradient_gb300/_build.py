"""Compile the CUDA library (csrc/*.cu over csrc/gq_kernels.cuh) into libgq.so, in-tree, and the
extension module through which Python calls its operators on tensors (csrc/gq_native.cpp).

Twelve translation units (the C ABI and the other kernels in gq.cu; the quantise launchers, one per
gradient type and scheme; the kernels of activations, 8-bit floating point and the optimizer) compiled in
parallel with one -gencode (sm_103a), then linked with the static CUDA runtime: the library depends on
nothing but the driver at load time.  -fmad=false keeps every fp32 operation of the gradient path and of the
optimizer a separately rounded IEEE operation (rounding decisions must be bit-identical to their definition);
the other units are compiled with contraction, and spell out the roundings that their codes depend on.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
UNITS = ["gq.cu", "gq_quant_f32_l.cu", "gq_quant_f32_e.cu", "gq_quant_bf16_l.cu",
         "gq_quant_bf16_e.cu", "gq_act.cu", "gq_layernorm_fwd.cu", "gq_layernorm_bwd.cu",
         "gq_wgrad.cu", "gq_fp8.cu", "gq_fp8_linear.cu", "gq_adamw.cu"]
CONTRACTED = {"gq_act.cu", "gq_layernorm_fwd.cu", "gq_layernorm_bwd.cu", "gq_wgrad.cu", "gq_fp8.cu",
              "gq_fp8_linear.cu"}
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgq.so")
# the same library with the kernels' bounds checks compiled in (-DGQ_DEBUG)
DEBUG_LIB = os.path.join(PKG, "libgq_debug.so")
NATIVE = os.path.join(CSRC, "gq_native.cpp")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "gq.h")])


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgq.so")
    return cand


def compile_command(unit: str, obj: str, extra=()) -> list:
    fmad = "-fmad=true" if unit in CONTRACTED else "-fmad=false"
    return [nvcc(), ARCH, "-O3", "-lineinfo", fmad, "-std=c++17", "-Xcompiler", "-fPIC",
            "-I" + os.path.join(ROOT, "include"), *extra, "-c", "-o", obj,
            os.path.join(CSRC, unit)]


def link_command(objs: list, out: str) -> list:
    return [nvcc(), ARCH, "-shared", "-o", out, *objs]


def native_path() -> str:
    """The extension module of this Python and torch (gq_native.cpp)."""
    import torch

    tag = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(PKG, "gq_native_%s.so" % tag)


def native_command(out: str) -> list:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return ["g++", "-O2", "-fPIC", "-shared", "-std=c++%d" % (20 if _torch_wants_cxx20() else 17),
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
            *["-isystem" + d for d in include_paths()], "-isystem" + cuda,
            "-isystem" + sysconfig.get_paths()["include"], "-I" + os.path.join(ROOT, "include"),
            NATIVE, "-o", out, "-L" + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch",
            "-lc10_cuda", "-lc10"]


def _torch_wants_cxx20() -> bool:
    import torch

    major, minor = (int("".join(c for c in v if c.isdigit())) for v in torch.__version__.split(".")[:2])
    return (major, minor) >= (2, 10)


def is_stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in sources())


def build_library(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Build libgq.so (debug: libgq_debug.so, with -DGQ_DEBUG) if missing or older than its
    sources, and beside it, where torch is installed, the extension module of the activation
    operators; return the library's path.  The library itself needs nvcc alone."""
    lib = DEBUG_LIB if debug else LIB
    building = None
    if not debug and importlib.util.find_spec("torch") is not None:
        native = native_path()
        if force or not os.path.exists(native) or any(
                os.path.getmtime(f) > os.path.getmtime(native)
                for f in (NATIVE, os.path.join(ROOT, "include", "gq.h"))):
            made = native + ".tmp.%d" % os.getpid()
            building = subprocess.Popen(native_command(made))
    try:
        _build_cuda(lib, force, verbose, debug)
    finally:
        if building is not None and building.wait() == 0:
            os.replace(made, native)
    if building is not None and building.returncode != 0:
        raise subprocess.CalledProcessError(building.returncode, "g++")
    return lib


def _build_cuda(lib: str, force: bool, verbose: bool, debug: bool) -> None:
    if force or is_stale(lib):
        os.makedirs(OBJ_DIR, exist_ok=True)
        extra = (("-Xptxas", "-v") if verbose else ()) + (("-DGQ_DEBUG",) if debug else ())
        tag = ".%d%s" % (os.getpid(), ".dbg" if debug else "")
        objs = [os.path.join(OBJ_DIR, u[:-3] + tag + ".o") for u in UNITS]
        tmp = lib + ".tmp" + tag
        try:
            procs = [subprocess.Popen(compile_command(u, o, extra)) for u, o in zip(UNITS, objs)]
            codes = [p.wait() for p in procs]
            if any(codes):
                raise subprocess.CalledProcessError(next(c for c in codes if c), "nvcc")
            subprocess.run(link_command(objs, tmp), check=True)
            os.replace(tmp, lib)
        finally:
            for f in objs + [tmp]:
                if os.path.exists(f):
                    os.remove(f)
