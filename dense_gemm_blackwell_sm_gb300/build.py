"""Build the CUDA library libdgbgemm.so in-tree (sm_103a only), and the Python
extensions that call include/ffn.h and include/quant.h of it.

Each translation unit under csrc/ is compiled by nvcc in parallel, then the
objects are linked into one shared library next to this file.  The CUDA
runtime is linked statically and the driver's tensor-map encoder is looked up
at run time, so loading the library needs no GPU.  The extensions (a C++ file each
against the installed torch's headers) lie next to it and load it from there.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdgbgemm.so")
CALLS = {"ffn_python.cpp": os.path.join(HERE, "_ffn_calls.so"),
         "quant_python.cpp": os.path.join(HERE, "_quant_calls.so")}

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in ("gemm.h", "ffn.h", "quant.h")]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-c", src, "-o", obj + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        os.replace(obj + ".tmp", obj)
    return obj


def _torch_root() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: the Python extension cannot be built")
    return spec.submodule_search_locations[0]


def _compile_calls(name: str) -> str:
    src, obj = os.path.join(CSRC, name), os.path.join(BUILD, name[:-4] + ".o")
    torch = _torch_root()
    if _stale(obj, [src, os.path.join(torch, "version.py")] + _headers()):
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
        cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE]
        for d in (sysconfig.get_paths()["include"], os.path.join(torch, "include"),
                  os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")):
            cmd += ["-isystem", d]
        r = subprocess.run(cmd + ["-c", src, "-o", obj + ".tmp"], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        os.replace(obj + ".tmp", obj)
    return obj


def _link_calls(name: str, obj: str) -> None:
    tmp, lib = CALLS[name] + ".tmp.%d" % os.getpid(), os.path.join(_torch_root(), "lib")
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, CALLS[name])


def build(force: bool = False, jobs: int | None = None, extra_flags=()) -> str:
    """Compile and link libdgbgemm.so and the extensions; returns the former's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if force:
        for f in os.listdir(BUILD):
            os.remove(os.path.join(BUILD, f))
    jobs = jobs or min(len(srcs) + len(CALLS), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = {name: ex.submit(_compile_calls, name) for name in CALLS}
        objs = list(ex.map(lambda s: _compile(s, extra_flags), srcs))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    for name, obj in calls.items():
        if force or _stale(CALLS[name], [obj.result()]):
            _link_calls(name, obj.result())
    return LIB


if __name__ == "__main__":
    print(build())
