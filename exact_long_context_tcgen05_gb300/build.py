"""Build libcqsa_gb300.so in-tree with nvcc for sm_103a (no CMake; translation units in parallel).

    python -m exact_long_context_tcgen05_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libcqsa_gb300.so")
SOURCES = ["attn_fwd.cu", "attn_bwd.cu", "merge.cu", "api.cu", "stream_driver.cu", "chunked_static.cu", "quorum.cu", "pool.cu", "stream_bwd.cu",
           "seq_api.cu", "kv_cache.cu", "attn_decode.cu", "attn_decode4.cu", "attn_seq.cu", "attn_select.cu"]
HEADERS = ["sm103_ptx.cuh", "cqsa_internal.h", "seq_common.cuh", "attn_common.cuh", "decode_common.cuh"]
BINDING = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _flags():
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                   "-Xptxas", "-warn-spills"]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_path() -> str:
    """The torch binding, one for each version of torch (it links to torch's own libraries)."""
    import torch
    return os.path.join(BUILD, f"cqsa_torch-{torch.__version__}.so")


def _binding_commands(obj: str, target: str) -> list:
    """Compiling the torch binding, and linking it to the library beside it and to torch."""
    import sysconfig

    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(at, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    cxx = os.environ.get("CXX", "g++")
    return [[cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in include),
             "-c", BINDING, "-o", obj],
            [cxx, "-shared", obj, LIB, "-o", target, "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
             "-ltorch_python"]]


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "cqsa.h")]
    objs, jobs = [], []
    cc = nvcc()
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *hdrs]):
            jobs.append([cc, *_flags(), "-c", s, "-o", o])
    bind = binding_path()
    bind_obj = bind.replace(".so", ".o")
    compile_bind, link_bind = _binding_commands(bind_obj, bind + f".{os.getpid()}.tmp")
    if force or _stale(bind_obj, [BINDING, os.path.join(ROOT, "include", "cqsa.h")]):
        jobs.append(compile_bind)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda cmd: subprocess.run(cmd, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"compiler failed: {' '.join(cmd)}")
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        r = subprocess.run([cc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs, "-cudart", "static"], capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
    if force or _stale(bind, [bind_obj, LIB]):
        r = subprocess.run(link_bind, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("linking the torch binding failed")
        os.replace(link_bind[link_bind.index("-o") + 1], bind)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
