"""Builds the CUDA library libgs_gb300.so in-tree with nvcc for sm_103a.

The translation units under csrc/ are compiled in parallel and linked into one shared object
with the C ABI of include/gs.h; csrc/bind.cpp becomes the Python module gs_bind.so, which calls it on
torch tensors (where torch is installed). The output goes to `_build/` beside this file.
"""
from __future__ import annotations

import concurrent.futures as cf
import dataclasses
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgs_gb300.so")
BIND = os.path.join(BUILD, "gs_bind.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgs_gb300.so")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch() -> tuple[str, str] | None:
    """torch's folder and version, without importing it; None where there is none."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    torch_dir = list(spec.submodule_search_locations)[0]
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            return torch_dir, f.read()
    except OSError:
        return torch_dir, ""


def _bind_commands(torch_dir: str, src: str, obj: str, out: str, nvcc: str) -> tuple[list[str], list[str]]:
    """The host compiler's commands for the Python module of the decoder operators' calls: compile, link."""
    torch_lib = os.path.join(torch_dir, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cxx = os.environ.get("CXX") or "g++"
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE] + [f for d in include for f in ("-isystem", d)] +
            ["-c", src, "-o", obj],
            [cxx, "-shared", obj, "-o", out, "-L" + torch_lib, "-L" + BUILD] +
            ["-l" + x for x in ("c10", "c10_cuda", "torch_cpu", "torch_cuda", "torch_python")] +
            ["-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN:" + torch_lib])


@dataclasses.dataclass
class _Bind:
    """What the Python module's build takes; made: what it is made with, kept beside the object."""
    obj: str
    tmp: str
    made: str
    compile: list[str]
    link: list[str]
    stale: bool


def _bind_jobs(nvcc: str, force: bool) -> _Bind | None:
    """None without torch, whose headers the module needs and the library does not. Another torch, Python or compiler than the
    module was made with makes it stale as much as its source does."""
    found = _torch()
    if found is None:
        return None
    src, obj, tmp = os.path.join(CSRC, "bind.cpp"), os.path.join(BUILD, "bind.o"), BIND + f".tmp{os.getpid()}"
    compile_, link = _bind_commands(found[0], src, obj, tmp, nvcc)
    made = " ".join(compile_) + "\n" + found[1]
    try:
        with open(obj + ".made") as f:
            same = f.read() == made
    except OSError:
        same = False
    return _Bind(obj, tmp, made, compile_, link, force or not same or _stale(obj, [src, os.path.join(INCLUDE, "gs.h")]))


def build_library(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC] + \
        list(extra_flags or [])
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([nvcc] + flags + ["-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed ({r.returncode}):\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    bind = _bind_jobs(nvcc, force)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        for msg in ex.map(run, ([bind.compile] if bind and bind.stale else []) + jobs):
            if verbose and msg:
                print(msg)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs +
            ["-Xlinker", "-rpath," + _cuda_lib_dir(nvcc)])
        os.replace(tmp, LIB)
    if bind and (bind.stale or _stale(BIND, [bind.obj])):
        run(bind.link)
        os.replace(bind.tmp, BIND)
        with open(bind.obj + ".made", "w") as f:
            f.write(bind.made)
    return LIB


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True))
