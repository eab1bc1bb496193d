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
    """The torch binding, one for each version of torch (it links to torch's own libraries) and interpreter."""
    import importlib.machinery

    import torch
    return os.path.join(BUILD, f"cqsa_torch-{torch.__version__}{importlib.machinery.EXTENSION_SUFFIXES[0]}")


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


def _run(cmd, verbose: bool) -> str:
    """Runs a compiler; returns what went wrong, or an empty string."""
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return f"{' '.join(cmd)}: {e}"
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    return f"compiler failed: {' '.join(cmd)}" if r.returncode else ""


class _Binding:
    """The torch binding: compiled beside the library's sources, linked to the library."""

    def __init__(self, force: bool, verbose: bool):
        self.verbose, self.target, self.failed = verbose, "", ""
        try:
            self.target = binding_path()
        except ImportError as e:
            self.failed = str(e)
            return
        self.obj, self.tmp = os.path.splitext(self.target)[0] + ".o", self.target + f".{os.getpid()}.tmp"
        self.compile, self.link = _binding_commands(self.obj, self.tmp)
        self.stale = force or _stale(self.obj, [BINDING, os.path.join(ROOT, "include", "cqsa.h")])

    def make_object(self):
        if not self.failed and self.stale:
            self.failed = _run(self.compile, self.verbose)

    def make(self):
        if not self.failed and (self.stale or _stale(self.target, [self.obj, LIB])):
            self.failed = _run(self.link, self.verbose)
            if not self.failed:
                os.replace(self.tmp, self.target)
        if self.failed:
            if os.path.exists(self.target):  # (one of older sources)
                os.remove(self.target)
            sys.stderr.write(f"the torch binding is not built, calls over a cache take longer on the host: {self.failed}\n")


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and beside it the torch binding where there are a torch and a C++ compiler: calls work without that one, more slowly on the host."""
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
    bind = _Binding(force, verbose)
    with cf.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        beside = ex.submit(bind.make_object)
        for wrong in list(ex.map(lambda cmd: _run(cmd, verbose), jobs)):
            if wrong:
                raise RuntimeError(wrong)
        beside.result()
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        wrong = _run([cc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs, "-cudart", "static"], verbose)
        if wrong:
            raise RuntimeError(wrong)
        os.replace(tmp, LIB)
    bind.make()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
