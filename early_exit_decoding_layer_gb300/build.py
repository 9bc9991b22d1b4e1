"""Builds libee.so (the CUDA kernels, runtime and C ABI) in-tree for sm_103a, and the
_binding extension module (the paged-cache operators' binding to PyTorch, with g++).

Each source is compiled in parallel, then linked into a shared library next to
this file.  libee.so needs nvcc alone.  The binding is left out where there is no
PyTorch, and an error in it is printed and stops nothing else: the operators' Python
functions raise where it is missing.  Usage: ``python -m early_exit_decoding_layer_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libee.so")
# named for this Python, so that another one does not load it
BINDING = os.path.join(HERE, "_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
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


def torch_dir():
    """The directory of PyTorch, None where there is none (it is not imported)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_version(t: str) -> str:
    """The text of PyTorch's version file."""
    with open(os.path.join(t, "version.py")) as f:
        return f.read()


def _binding_commands(cc: str, t: str, obj: str, out: str):
    """(compile, link) of the binding."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(cc)))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    version = re.search(r"^__version__ = '([^']*)'", _torch_version(t), re.M).group(1)
    compile_ = [cxx, "-O2", "-fPIC", "-std=c++17", "-fvisibility=hidden", '-DEE_TORCH_VERSION="%s"' % version,
                *["-I" + i for i in inc], "-c", BINDING_SRC, "-o", obj]
    lib = os.path.join(t, "lib")
    link = [cxx, "-shared", "-o", out, obj, "-L" + os.path.dirname(LIB), "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
            "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


class _Binding:
    """The binding's part of a build.  `stamp` says what the binding on disk was built with:
    the commands and PyTorch's version file, in which neither source nor header shows."""

    def __init__(self, cc: str, hdrs, force: bool):
        self.dir = torch_dir()
        self.compile = None
        if self.dir is None:
            return
        obj, self.stamp = os.path.join(BUILD, "ee_binding.o"), os.path.join(BUILD, "ee_binding.stamp")
        compile_, self.link = _binding_commands(cc, self.dir, obj, BINDING)
        self.want = "\n".join([" ".join(compile_), " ".join(self.link), sys.version, _torch_version(self.dir)])
        have = ""
        if os.path.exists(self.stamp):
            with open(self.stamp) as f:
                have = f.read()
        if force or have != self.want or _stale(obj, [BINDING_SRC] + hdrs) or _stale(BINDING, [obj]):
            self.compile = compile_

    def finish(self, compiled):
        """Links what `compiled` (the finished compile process) made; True if the binding is there."""
        if os.path.exists(self.stamp):
            os.remove(self.stamp)
        tmp = BINDING + ".%d.tmp" % os.getpid()
        r = compiled
        if r.returncode == 0:
            r = _run([tmp if x == BINDING else x for x in self.link])[1]
        if r.returncode != 0:
            sys.stderr.write("the binding to PyTorch was not built (libee.so is not affected):\n" + r.stdout + r.stderr)
            if os.path.exists(BINDING):
                os.remove(BINDING)  # it is not of these sources
            return False
        os.replace(tmp, BINDING)
        with open(self.stamp, "w") as f:
            f.write(self.want)
        return True


def _run(cmd):
    try:
        return cmd, subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return cmd, subprocess.CompletedProcess(cmd, 1, "", "%s: %s\n" % (cmd[0], e))


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

    binding = _Binding(cc, hdrs, force)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        bound = ex.submit(_run, binding.compile) if binding.compile else None
        for cmd, r in ex.map(_run, jobs):
            if verbose or ptxas_info or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("compilation of %s failed" % cmd[-3])
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".%d.tmp" % os.getpid()
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link of libee.so failed")
        os.replace(tmp, LIB)
    if bound:
        binding.finish(bound.result()[1])
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                ptxas_info="--ptxas" in sys.argv))
