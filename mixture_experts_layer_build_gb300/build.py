"""Build ``libmok.so`` in-tree with nvcc for sm_103a (one -gencode, translation units in parallel), and the compiled
part of the Python binding, ``_mok_bind.so``, with g++."""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmok.so")
BIND = os.path.join(HERE, "_mok_bind.so")
BIND_TARGET = os.path.join(BUILD, "mok_bind.target")  # what BIND was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
SOURCES = ["mok_api.cu", "mok_sched.cu", "mok_move.cu", "mok_gemm_fwd.cu", "mok_gemm_dgrad.cu", "mok_gemm_wgrad.cu",
           "mok_router.cu", "mok_noalloc.cu", "mok_norm.cu",
           "mok_ffn.cu", "mok_ffn_tile.cu", "mok_ffn_pair.cu", "mok_ffn_row.cu",
           "mok_route.cu", "mok_fp8.cu", "mok_fp8_quant.cu", "mok_fp8_tile.cu", "mok_fp8_pair.cu"]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    import importlib.util
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def bind_target() -> str:
    """What _mok_bind.so is built for: torch's inlined accessors and Python's ABI are in it.  (torch's version from its
    own file: the build does not import torch.)"""
    text = open(os.path.join(_torch_dir(), "version.py")).read()
    version = re.search(r"^__version__ = ['\"](.+?)['\"]", text, re.M).group(1)
    return f"torch {version}, python {sys.version_info.major}.{sys.version_info.minor}"


def _bind_commands() -> list:
    """[compile, link] of _mok_bind.so against this machine's torch; it finds libmok.so beside it."""
    import sysconfig
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(NVCC))
    obj = os.path.join(BUILD, "mok_bind.o")
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    cxx = os.environ.get("CXX", "g++")
    return [[cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{i}" for i in inc),
             f'-DMOK_BUILT_FOR="{bind_target()}"', "-c", os.path.join(CSRC, "mok_bind.cpp"), "-o", obj],
            [cxx, "-shared", obj, "-o", BIND + f".tmp{os.getpid()}", f"-L{HERE}", "-l:libmok.so", "-Wl,-rpath,$ORIGIN",
             f"-L{os.path.join(torch, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]]


def bind_stale() -> bool:
    """Whether _mok_bind.so has to be compiled: sources that changed, or another torch or Python than it is for."""
    compile_bind = _bind_commands()[0]
    if _stale(compile_bind[-1], [compile_bind[-3], os.path.join(INCLUDE, "mok.h"), __file__]):
        return True
    return not os.path.exists(BIND_TARGET) or open(BIND_TARGET).read() != bind_target()


def build(verbose: bool = False, extra=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "mok.h"))
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if _stale(o, [s, *headers, __file__]):
            jobs.append([NVCC, *ARCH, *FLAGS, *(extra or []), "-c", s, "-o", o])
    compile_bind, link_bind = _bind_commands()
    if bind_stale():
        jobs.append(compile_bind)
    failed = []
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            res = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, res):
            if verbose or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                failed.append(cmd)
    for cmd in failed:
        if cmd is not compile_bind:  # the library is linked without the binding, which the routed layer does not need
            raise RuntimeError(f"the compiler failed on {cmd[-3]}")
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cudalib = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "lib64")
        r = subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", f"-rpath,{cudalib}", "-o", tmp,
                            *objs], capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libmok.so failed")
        os.replace(tmp, LIB)
    if failed:
        raise RuntimeError(f"the compiler failed on {compile_bind[-3]}")
    if _stale(BIND, [compile_bind[-1]]):
        r = subprocess.run(link_bind, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of _mok_bind.so failed")
        os.replace(BIND + f".tmp{os.getpid()}", BIND)
        with open(BIND_TARGET, "w") as f:
            f.write(bind_target())
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
