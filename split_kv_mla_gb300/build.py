"""Build libmla.so in-tree: every ``csrc/*.cu`` compiled for sm_103a in parallel,
then linked into ``split_kv_mla_gb300/_build/libmla.so``; beside it the extension
module of mla.py's argument checks (``csrc/mla_binding.cpp``).

Run ``python -m split_kv_mla_gb300.build`` (or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmla.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _cuda_lib_dir() -> str:
    nvcc = os.path.realpath(_nvcc())
    root = os.path.dirname(os.path.dirname(nvcc))
    for sub in ("lib64", "lib", "targets/sbsa-linux/lib", "targets/x86_64-linux/lib"):
        p = os.path.join(root, sub)
        if os.path.isdir(p):
            return p
    return os.path.join(root, "lib64")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, obj: str, extra) -> None:
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)


def binding_path() -> str:
    """The extension module's file, named after the torch and Python it is built for."""
    import torch
    return os.path.join(BUILD, "torch-" + torch.__version__,
                        "mla_binding" + sysconfig.get_config_var("EXT_SUFFIX"))


def build_binding(force: bool = False) -> str:
    """Compile csrc/mla_binding.cpp against this torch; returns the module's path."""
    import torch
    path = binding_path()
    src = os.path.join(CSRC, "mla_binding.cpp")
    if not force and not _stale(path, [src, *_headers()]):
        return path
    os.makedirs(os.path.dirname(path), exist_ok=True)
    tdir = os.path.dirname(torch.__file__)
    tlib = os.path.join(tdir, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(tdir, "include"),
           "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"),
           "-isystem", sysconfig.get_paths()["include"], src, "-o", tmp, "-L", tlib,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + tlib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for mla_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra=(), build_dir: str = BUILD) -> str:
    """Compile every csrc/*.cu (extra nvcc flags appended) into build_dir and
    link build_dir/libmla.so, and for the standard build_dir the extension
    module; returns the library's path."""
    lib = os.path.join(build_dir, "libmla.so")
    os.makedirs(build_dir, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    jobs = []
    objs = []
    for src in sources:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *headers]):
            jobs.append((src, obj))
    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        futs = [ex.submit(_compile, s, o, list(extra)) for s, o in jobs]
        if build_dir == BUILD:
            futs.append(ex.submit(build_binding, force))
        for f in futs:
            f.result()
    if force or jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        libdir = _cuda_lib_dir()
        cmd = [_nvcc(), *ARCH, "-shared", "-cudart=shared", "-o", tmp, *objs,
               "-L", libdir, "-Xlinker", "-rpath=" + libdir]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if verbose:
        print(lib)
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
