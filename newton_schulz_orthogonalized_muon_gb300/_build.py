"""Build libmuon_gb300.so in-tree with nvcc for sm_103a (GB300), and the
extension module that calls it on torch tensors.

The translation units compile in parallel; the shared library links the CUDA
runtime statically and resolves the tensor-map encoder from the driver at run
time, so it needs no -lcuda.  The module (host code) links that library and
torch's; its object's name carries torch's version and the link command is
kept, so that another torch gets another build.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libmuon_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["muon_api.cu", "kernels_tc.cu", "kernels_tc2.cu", "kernels_elem.cu", "kernels_simt.cu", "noalloc.cu",
           "ops_api.cu", "op_norm.cu", "op_act8.cu", "op_wgrad.cu", "op_attn_fwd.cu", "op_attn_bwd.cu"]
HEADERS = ["common.cuh", "internal.h", "tc_common.cuh", "launch_opts.h", "handle.h", "op_common.cuh", "op_attn.cuh"]
MODULE_SOURCE = os.path.join(CSRC, "torch_ops.cpp")
MODULE_PATH = os.path.join(HERE, "_torch_ops.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")


def _module_commands(nvcc: str):
    """(object, compile command, link command) of the extension module."""
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    dirs = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda, INCLUDE]
    obj = os.path.join(BUILD_DIR, f"torch_ops-{torch.__version__}.o")
    cxx = shutil.which("g++") or "c++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *[f for d in dirs for f in ("-isystem" if d != INCLUDE else "-I", d)], "-c", MODULE_SOURCE, "-o", obj]
    link = [cxx, "-shared", obj, "-o", MODULE_PATH, LIB_PATH, "-Wl,-rpath,$ORIGIN", "-L", os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return obj, compile_, link


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every translation unit (in parallel), link the library and then
    the extension module.  Returns the path of the shared library."""
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "muon.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o])
    lib_jobs = len(jobs)
    mod_error = None
    try:
        mod_obj, mod_compile, mod_link = _module_commands(nvcc)
        if force or _stale(mod_obj, [MODULE_SOURCE, os.path.join(INCLUDE, "muon.h")]):
            jobs.append(mod_compile)
    except ImportError as e:                     # no torch: the library is built all the same
        mod_error = e

    def run(cmd):
        """None, or the command's failure."""
        if verbose:
            print(" ".join(cmd), flush=True)
        try:
            r = subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:
            return RuntimeError(f"compilation failed:\n{' '.join(cmd)}\n{e}")
        if verbose and r.returncode == 0 and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return RuntimeError(f"compilation failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}") if r.returncode else None

    def need(error):
        if error is not None:
            raise error

    errors = []
    if jobs:
        with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            errors = list(ex.map(run, jobs))
    for e in errors[:lib_jobs]:
        need(e)
    if force or lib_jobs or _stale(LIB_PATH, objs):
        need(run([nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-Xlinker", f"-soname={LIB_NAME}", "-o", LIB_PATH]))
    # then the module: the library does not depend on torch or on its headers
    need(mod_error)
    for e in errors[lib_jobs:]:
        need(e)
    # what the module was linked from: an older object of another torch's is not newer than it
    stamp = os.path.join(BUILD_DIR, "torch_ops.link")
    last = open(stamp).read() if os.path.exists(stamp) else None
    if force or last != " ".join(mod_link) or _stale(MODULE_PATH, [mod_obj, LIB_PATH]):
        need(run(mod_link))
        with open(stamp, "w") as f:
            f.write(" ".join(mod_link))
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
