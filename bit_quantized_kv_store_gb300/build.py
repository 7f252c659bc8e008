"""Build libkvq.so (the CUDA kernels + C ABI) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel, then linked into
``bit_quantized_kv_store_gb300/_build/libkvq.so``; the compiled part of the Python
binding becomes ``_kvq_calls.so`` beside it, where there is a torch to bind to.  A
unit is rebuilt only when its source or a header is newer than its object file, the
binding also for another interpreter or torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
# KVQ_SANITIZE=1: a separate build of the host code with AddressSanitizer and
# UndefinedBehaviorSanitizer, for checking the C ABI's argument validation on
# the CPU (device code as PTX only: that build never launches a kernel).
SANITIZE = os.environ.get("KVQ_SANITIZE") == "1"
BUILD = os.path.join(PKG, "_build_san" if SANITIZE else "_build")
LIB = os.path.join(BUILD, "libkvq.so")
CALLS = os.path.join(BUILD, "_kvq_calls.so")  # csrc/binding.cpp
CALLS_STAMP = CALLS + ".for"

ARCH = ["-gencode", "arch=compute_103a,code=compute_103a" if SANITIZE else "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{os.path.join(ROOT, 'include')}"]
SAN_FLAGS = ["-Xcompiler", "-fsanitize=address", "-Xcompiler", "-fsanitize=undefined",  # (-Xcompiler splits at commas)
             "-Xcompiler", "-fno-sanitize-recover=undefined", "-Xcompiler", "-fno-omit-frame-pointer"]
if SANITIZE:
    FLAGS = FLAGS + SAN_FLAGS
# The store computes codes that must be bit-exact: no fused multiply-adds there.
PER_FILE = {"store.cu": ["-fmad=false"], "tq4.cu": ["-fmad=false"], "norm_rope.cu": ["-fmad=false"],
            "latent.cu": ["-fmad=false"]}


def _tool_env():
    """The environment for the compilers: without a preloaded sanitizer runtime
    (a sanitized test process preloads one, and nvcc's own tools crash under it)."""
    return {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers_mtime():
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _headers_mtime()):
        return obj, ""
    cmd = [_nvcc(), *ARCH, *FLAGS, *PER_FILE.get(os.path.basename(src), []), "-c", src, "-o", obj + ".tmp"]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True, env=_tool_env())
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, r.stderr


def _made_for(torch):
    """What the compiled part of the binding was made for: an interpreter and a torch."""
    return f"{sys.version}\n{sysconfig.get_config_var('SOABI')}\n{torch.__version__} {torch.__file__}\n"


def _build_calls():
    """The compiled part of the Python binding, against the installed torch.  Without
    torch there is no binding to build: the library serves programs of the C ABI alone."""
    try:
        import torch
    except ImportError:
        return
    src, header = os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "kvq.h")
    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    made_for = _made_for(torch)
    if os.path.exists(CALLS) and os.path.exists(CALLS_STAMP):
        with open(CALLS_STAMP) as f:
            same = f.read() == made_for
        if same and os.path.getmtime(CALLS) >= max(os.path.getmtime(p) for p in (src, header)):
            return
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-o", tmp, src,
           f"-I{sysconfig.get_paths()['include']}", f"-I{tdir}/include", f"-I{tdir}/include/torch/csrc/api/include",
           f"-I{cuda}/include", f"-L{tdir}/lib", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10",
           f"-Wl,-rpath,{tdir}/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True, env=_tool_env())
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(CALLS_STAMP):
        os.remove(CALLS_STAMP)  # (never the new module's stamp beside the old module)
    os.replace(tmp, CALLS)
    with open(tmp, "w") as f:
        f.write(made_for)
    os.replace(tmp, CALLS_STAMP)


def build(verbose_ptxas=False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        calls = ex.submit(_build_calls)
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    if verbose_ptxas:
        for _, log in results:
            if log:
                print(log)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, *(SAN_FLAGS if SANITIZE else [])]
        r = subprocess.run(cmd, capture_output=True, text=True, env=_tool_env())
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    calls.result()  # (its failure is raised with the library in place)
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv))
