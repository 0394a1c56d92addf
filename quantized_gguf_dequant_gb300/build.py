"""Build libqmm.so (the CUDA library behind include/qmm.h) in-tree.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into one shared object next to this file; the native part of the Python binding
(host code) is compiled beside them where torch is installed.  `python -m
quantized_gguf_dequant_gb300.build` does the same from a shell.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqmm.so")
NATIVE = os.path.join(HERE, "_native.so")  # the binding of the decode-step calls
BINDING = "binding.cpp"
SOURCES = ["qmm_api.cu", "dequant.cu", "gemv.cu", "gemv_tc.cu", "qmm_noalloc.cu", "moe.cu", "gemm_tc.cu", "tmap.cu", "gemv_batched.cu", "formats.cu", "gemv_m1.cu", "q8k.cu", "formats_fast.cu", "gemv_tc5.cu", "moe_q8.cu", "decode_api.cu", "kv_append.cu", "attn_decode.cu", "attn_f16.cu", "attn_bf16.cu", "attn_q8.cu", "logits.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-ftz=false", "-prec-div=true",
                   "-prec-sqrt=true", "-fmad=true", "-Xcompiler", "-fPIC",
                   "-Xcompiler", "-fvisibility=hidden", "-I" + os.path.join(ROOT, "include")]


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), "-c", os.path.join(CSRC, src), "-o", obj] + _flags()
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _torch_dir():
    """Where torch is installed, or None (the C library does not need it)."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _build_native(torch_dir: str) -> str:
    """csrc/binding.cpp against torch's headers (host code only)."""
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = NATIVE + f".tmp.{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=1",
           "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(torch_dir, "include"),
           "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC, BINDING), "-o", tmp, "-L" + os.path.join(torch_dir, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"the Python binding needs a C++ compiler: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def _build_library(verbose_ptxas: bool) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    tmp = LIB + f".tmp.{os.getpid()}"
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    deps = [os.path.join(CSRC, f) for f in sources]
    deps += [os.path.join(ROOT, "include", "qmm.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library, and where torch is installed the native part of the binding.
    The library is there also when that part fails."""
    force = force or verbose_ptxas
    torch_dir = _torch_dir()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        native = None
        if torch_dir and (force or _stale(NATIVE, [BINDING])):
            native = ex.submit(_build_native, torch_dir)
        if force or _stale(LIB, [f for f in os.listdir(CSRC) if f != BINDING]):
            _build_library(verbose_ptxas)
        if native:
            native.result()
    if not torch_dir:
        print("torch is not installed: the Python binding's native part was not built",
              file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
