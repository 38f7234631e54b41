"""Build libemufp8.so (the GEMM library) and libemupeaks.so (the instruction-rate
microbenchmark bench.py divides by) in-tree with nvcc for sm_103a (GB300), and the
operators' torch-facing calls (_ops_torch.so) with the host compiler.

    python -m bit_exact_fp8_gb300.build [--force]

One -gencode, no cmake; the two libraries and the GEMM library's translation units
compile in parallel, and each library is rebuilt only when one of its sources or
headers is newer.
"""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libemufp8.so")
PEAKS_LIB = os.path.join(PKG, "libemupeaks.so")
OPS_LIB = os.path.join(PKG, "_ops_torch.so")
SOURCES = [os.path.join(CSRC, f) for f in ("emu_api.cu", "ops_norm.cu", "ops_int8.cu",
                                           "ops_logprob.cu", "ops_block_quant.cu", "ops_block_mm.cu")]
PEAKS_SOURCES = [os.path.join(CSRC, "emu_peaks.cu")]
PEAKS_DEPS = PEAKS_SOURCES + [os.path.join(INCLUDE, "emu_peaks.h")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] \
    + [os.path.join(INCLUDE, "emu_fp8.h")]

#: what stands before built_for() in the operators' extension
OPS_MARK = "emu operators built for "
OPS_SOURCES = [os.path.join(CSRC, "ops_torch.cpp")]
OPS_DEPS = OPS_SOURCES + [os.path.join(CSRC, "ops_torch_block.h"), os.path.join(INCLUDE, "emu_fp8.h")]

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "--threads", "0", "-I" + INCLUDE, "-I" + CSRC]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libemufp8")


def _up_to_date(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in deps)


def built_for() -> str:
    """What the operators' extension is tied to, and is made anew for: torch and Python (and with
    Python's tag the machine)."""
    return f"torch {importlib.metadata.version('torch')}, {sysconfig.get_config_var('SOABI')}"


def ops_built_for(lib: str) -> str:
    """What the extension at this path was built for, "" if it does not say: read from the file, as
    an extension of another torch may not survive its loading."""
    mark = OPS_MARK.encode()
    with open(lib, "rb") as f:
        data = f.read()
    at = data.find(mark)
    return data[at + len(mark):data.index(b"\0", at)].decode(errors="replace") if at >= 0 else ""


def _ops_up_to_date() -> bool:
    return _up_to_date(OPS_LIB, OPS_DEPS) and ops_built_for(OPS_LIB) == built_for()


def up_to_date() -> bool:
    return _up_to_date(LIB, DEPS) and _up_to_date(PEAKS_LIB, PEAKS_DEPS) and _ops_up_to_date()


def ops_commands(out: str) -> "tuple[list, list]":
    """The host compiler's commands that make the operators' extension from its source: one
    that compiles, and one that links it to torch and to the libemufp8 beside it."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    obj = out + ".o"
    includes = [INCLUDE] + include_paths() + [os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    compile_ += [f'-DEMU_OPS_BUILT_FOR="{OPS_MARK}{built_for()}"']
    compile_ += [f"-I{d}" for d in includes] + ["-c"] + OPS_SOURCES + ["-o", obj]
    link = ["g++", "-shared", obj, "-o", out, f"-L{PKG}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    link += [f"-L{d}" for d in library_paths()] + ["-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile whichever of the two libraries and the operators' extension is stale; returns the
    GEMM library's path.  Each is put in place as soon as it is made, whatever becomes of the
    others (the libraries need nvcc alone); what could not be made is raised at the end."""
    jobs = []
    for lib, srcs, deps in ((LIB, SOURCES, DEPS), (PEAKS_LIB, PEAKS_SOURCES, PEAKS_DEPS)):
        if force or not _up_to_date(lib, deps):
            tmp = lib + f".tmp{os.getpid()}"
            cmd = [nvcc_path()] + NVCC_FLAGS + srcs + ["-o", tmp]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            jobs.append((lib, tmp, subprocess.Popen(cmd)))
    failed, ops_proc = [], None
    ops_tmp = OPS_LIB + f".tmp{os.getpid()}"
    try:
        ops_stale = force or not _ops_up_to_date()
    except ImportError:                                      # no torch: said below
        ops_stale = True
    if ops_stale:
        try:
            ops_compile, ops_link = ops_commands(ops_tmp)
            if verbose:
                print(" ".join(ops_compile), file=sys.stderr)
            ops_proc = subprocess.Popen(ops_compile)
        except (ImportError, OSError) as e:                  # no torch, or no host compiler
            failed.append(f"{OPS_LIB}: {e}")
    for lib, tmp, proc in jobs:
        if proc.wait() == 0:
            os.replace(tmp, lib)
        else:
            failed.append(lib)
    if ops_proc is not None:
        if ops_proc.wait() == 0 and os.path.exists(LIB) and subprocess.run(ops_link).returncode == 0:
            os.replace(ops_tmp, OPS_LIB)
        else:
            failed.append(OPS_LIB)
        if os.path.exists(ops_tmp + ".o"):
            os.remove(ops_tmp + ".o")
    if failed:
        raise subprocess.CalledProcessError(1, f"nvcc or g++ ({', '.join(failed)})")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
