"""Builds libee.so (the CUDA kernels, runtime and C ABI) in-tree for sm_103a, and
_binding.so (the paged-cache operators' binding to PyTorch, with g++).

Each source is compiled in parallel, then linked into a shared library next to
this file.  Usage: ``python -m early_exit_decoding_layer_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libee.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "ee_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]
# EE_NVCC_EXTRA="-DEE_CHECKED" builds the self-checking debug variant of the kernels.
NVCC_FLAGS += os.environ.get("EE_NVCC_EXTRA", "").split()


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put CUDA's bin directory on PATH")


def torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("PyTorch not found: the binding is built against its headers")
    return os.path.dirname(spec.origin)


def _binding_commands(cc: str, obj: str, out: str):
    """(compile, link) of _binding.so."""
    t, cuda = torch_dir(), os.path.dirname(os.path.dirname(os.path.realpath(cc)))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_ = [cxx, "-O2", "-fPIC", "-std=c++17", "-fvisibility=hidden", *["-I" + i for i in inc], "-c", BINDING_SRC, "-o", obj]
    lib = os.path.join(t, "lib")
    link = [cxx, "-shared", "-o", out, obj, "-L" + HERE, "-l:libee.so", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(HERE, "..", "include", "*.h")))


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    cc = nvcc()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    bobj = os.path.join(BUILD, "ee_binding.o")
    bcompile, _ = _binding_commands(cc, bobj, BINDING)
    bnew = force or _stale(bobj, [BINDING_SRC] + hdrs)
    if bnew:
        jobs.append(bcompile)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or ptxas_info or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("compilation of %s failed" % cmd[-3])
    if force or len(jobs) > bnew or _stale(LIB, objs):
        tmp = LIB + ".%d.tmp" % os.getpid()
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link of libee.so failed")
        os.replace(tmp, LIB)
    if bnew or _stale(BINDING, [bobj]):
        tmp = BINDING + ".%d.tmp" % os.getpid()
        cmd = _binding_commands(cc, bobj, tmp)[1]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link of _binding.so failed")
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                ptxas_info="--ptxas" in sys.argv))
