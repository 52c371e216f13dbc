"""Build libattn.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and
_quick.so (csrc/binding.cpp, the binding's quick way into it) with g++ against
the installed torch.

Each translation unit is compiled in parallel into ``_build/`` and linked into
``exact_attention_forward_06_gb300/``.  Rebuilds only when a source or header is
newer than the libraries, or when _quick.so was built against another torch or
Python (_quick.abi says which).  Usable as a script:
``python -m exact_attention_forward_06_gb300.build [--force] [--verbose]``.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libattn.so")
QUICK = os.path.join(PKG, "_quick.so")
QUICK_ABI = os.path.join(PKG, "_quick.abi")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                     "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (needs the CUDA 13 toolkit)")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def abi_tag() -> str:
    """What _quick.so, unlike libattn.so, is bound to: the installed torch's C++ interface and the Python it runs in."""
    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"{sysconfig.get_config_var('SOABI')}")


def built_abi():
    """abi_tag() of the torch and Python that _quick.so was built against; None if it was not built."""
    try:
        with open(QUICK_ABI) as f:
            return f.read()
    except OSError:
        return None


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(QUICK)) or built_abi() != abi_tag():
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(QUICK))
    deps = sources() + [os.path.join(CSRC, "binding.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def _compile(src: str, extra, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def _run(cmd, what: str, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_binding(verbose: bool):
    """binding.cpp as an object, and what links it to torch."""
    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    obj = os.path.join(BUILD_DIR, "binding.o")
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE] + [x for i in inc for x in ("-isystem", i)] + \
        [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", os.path.join(CSRC, "binding.cpp"),
         "-o", obj]
    _run(cmd, "g++ on binding.cpp", verbose)
    lib = os.path.join(base, "lib")
    return [obj, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the sources under csrc/ and link libattn.so and _quick.so; returns libattn.so's path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs +
         ["-Xlinker", "-rpath=/usr/local/cuda/lib64"], "link", verbose)
    os.replace(tmp, LIB)
    tmp = QUICK + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp] + binding.result() + ["-L", PKG, "-l:libattn.so", "-Wl,-rpath,$ORIGIN"],
         "link of the binding", verbose)
    if os.path.exists(QUICK_ABI):
        os.remove(QUICK_ABI)
    os.replace(tmp, QUICK)
    with open(QUICK_ABI, "w") as f:
        f.write(abi_tag())
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    verbose = "--verbose" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force or bool(extra), verbose=verbose or bool(extra), extra=extra))
