"""Build ``libflash_mca.so`` in-tree with nvcc for sm_103a.

The translation units compile in parallel (the C-ABI layer, the SIMT kernels,
the tensor-core kernels and the layer norm among them) and link into one shared
library next to this file.  The CUDA runtime is linked statically and the driver's
tensor-map encoder is looked up at run time, so the library loads on a machine
without a GPU driver (only calls that touch the device need one).  The Python
module with the training operators' wrappers (host code over torch's headers, by
g++) compiles beside them; where it cannot, the rest of the package works.

The package runs ``build()`` on import (a no-op when both are newer than their
sources); ``python -m flash_mixed_chunk_gb300.build [--force] [-v]`` runs it by
hand.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libflash_mca.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_STAMP = os.path.join(PKG, "_binding.stamp")

SOURCES = ["api.cpp", "simt.cu", "tc.cu", "noalloc.cu", "decode.cu", "backward.cu",
           "api_train.cpp", "norm.cu", "api_serve.cpp", "decay.cu", "beam.cu"]
HEADERS = ["launch.h", "ptx.cuh", "tc_common.cuh", "tc_prep.cuh", "tc_attn.cuh", "tc_fused.cuh", "tc_walk.cuh", "tc_pair.cuh", "tc_gemm.cuh", "tc_bgemm.cuh", "tc_bwd.cuh", "tc_backward.cuh",
           "tg_plan.h", "tc_tgemm.cuh", "tc_train.cuh", "decay.cuh",
           "tc_decay.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libflash_mca.so")


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] +
                  [os.path.join(INCLUDE, "flash_mca.h"), os.path.abspath(__file__)])


def _binding_against() -> str:
    """What the module is compiled against: another Python or torch may lay out its
    objects otherwise, whatever the files' times say."""
    import torch
    return f"{sys.version}\n{torch.__version__} {torch._C._GLIBCXX_USE_CXX11_ABI}\n"


def _binding_stale() -> bool:
    try:
        with open(BINDING_STAMP) as f:
            if f.read() != _binding_against():
                return True
    except OSError:
        return True
    return _older(BINDING, [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "flash_mca.h"),
                            os.path.abspath(__file__)])


def _binding_compile():
    """Starts the compiler on binding.cpp (host code over torch's C++ headers)."""
    import torch
    os.makedirs(BUILD, exist_ok=True)
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    paths = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"),
             sysconfig.get_paths()["include"],
             os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for p in paths for x in ("-isystem", p)], "-c", os.path.join(CSRC, "binding.cpp"),
           "-o", os.path.join(BUILD, "binding.o")]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _binding_link() -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, os.path.join(BUILD, "binding.o"), "-L", PKG,
                    "-l:libflash_mca.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python",
                    "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_against())


class BindingError(RuntimeError):
    """The library is there, the module with the training operators' wrappers is not."""


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is out of date; raises BindingError where that fails for the
    module alone."""
    lib, binding = force or _stale(), force or _binding_stale()
    binding_proc = binding_error = None
    if binding:
        try:
            binding_proc = _binding_compile()
        except Exception as exc:  # no host compiler, nowhere to write
            binding_error = exc
    if lib:
        _build_library(verbose)
    if binding_proc is not None:
        out = binding_proc.communicate()[0].decode(errors="replace")
        if verbose or binding_proc.returncode != 0:
            sys.stdout.write(out)
        try:
            if binding_proc.returncode != 0:
                raise RuntimeError("compilation failed for binding.cpp")
            _binding_link()
        except Exception as exc:
            binding_error = exc
    if binding_error is not None:
        raise BindingError(f"{BINDING} could not be built (it needs g++, Python's and torch's "
                           f"headers): {binding_error}") from binding_error
    return LIB


def _build_library(verbose: bool) -> None:
    cc = nvcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.rsplit(".", 1)[0] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cu"):
            cmd += ["-Xptxas", "-v"] if verbose else []
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stdout.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
