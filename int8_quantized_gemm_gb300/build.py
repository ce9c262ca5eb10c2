"""Build the CUDA library libq8.so in-tree for sm_103a.

Each .cu file is compiled separately (in parallel) and linked into one shared
library with the C ABI of include/q8.h. Beside it, one small module of the host compiler against the
installed PyTorch: the common calls of the 4-bit operators (csrc/q8_calls.cpp), without which the binding
makes them itself. Run `python -m int8_quantized_gemm_gb300.build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libq8.so")
SOURCES = ["q8_api.cu", "q8_quant.cu", "q8_gemm_mma.cu", "q8_gemm_tc.cu", "q8_gemv_tc.cu", "q8_gemv_mma.cu", "q8_gemm_tc2.cu",
           "q8_host.cu", "q8_fp8_api.cu", "q8_fp8_quant.cu", "q8_fp8_gemm.cu", "q8_moe.cu",
           "q8_fp4_api.cu", "q8_fp4_quant.cu", "q8_fp4_gemm.cu"]
CALLS_SOURCE = "q8_calls.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libq8.so")


def calls_path() -> str:
    """The module of the common calls, for this interpreter and PyTorch."""
    tag = f"{sys.implementation.cache_tag}_torch_{torch.__version__}"
    return os.path.join(OUT_DIR, "_q8_calls_" + "".join(c if c.isalnum() else "_" for c in tag) + ".so")


def _build_calls() -> str:
    """Compiles it to calls_path() + ".tmp". Returns why it could not be compiled (the binding works without it), or an empty
    string."""
    out = calls_path()
    torch_dir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    cc = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cc:
        return "no host compiler"
    cmd = [cc, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I", inc,
           "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           os.path.join(CSRC, CALLS_SOURCE), "-o", out + ".tmp", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{lib}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return str(e)
    return "" if r.returncode == 0 else r.stderr[-2000:] or f"{cc}: status {r.returncode}"


def _install(lib: str, why: str):
    """Puts a new library in place, and its module of the common calls where that could be compiled (`why` is empty). A module calls
    the C ABI that it was compiled against, so those of the library before, for other interpreters too, go first."""
    for old in glob.glob(os.path.join(glob.escape(OUT_DIR), "_q8_calls_*.so")) + [calls_path() + ".none"]:
        if os.path.exists(old):
            os.remove(old)
    os.replace(lib, LIB)
    if why:
        open(calls_path() + ".none", "w").close()
        sys.stderr.write(f"{CALLS_SOURCE} was not built, the binding makes these calls itself: {why}\n")
    else:
        os.replace(calls_path() + ".tmp", calls_path())


def _flags(verbose: bool):
    f = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-fmad=false",
         "-I", os.path.join(ROOT, "include"), *ARCH]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _stale() -> bool:
    made = [p for p in (calls_path(), calls_path() + ".none") if os.path.exists(p)]   # .none: it could not be compiled here
    if not os.path.exists(LIB) or not made:
        return True
    t = min(os.path.getmtime(LIB), max(os.path.getmtime(p) for p in made))
    headers = ["q8_internal.h", "q8_tc_ptx.cuh", "q8_fp8.h", "q8_fp8_ptx.cuh", "q8_tiles.cuh", "q8_loads.cuh", "q8_silu.cuh", "q8_fp4.h",
               "q8_fp4_ptx.cuh"]
    deps = [os.path.join(CSRC, s) for s in SOURCES + headers + [CALLS_SOURCE]] + [os.path.join(ROOT, "include", "q8.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *_flags(verbose), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_build_calls)
        for obj, log in ex.map(compile_one, SOURCES):
            objs.append(obj)
            if verbose and log:
                sys.stderr.write(log)
        why = calls.result()
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _install(tmp, why)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
