"""Builds libkvevict.so in-tree with nvcc for sm_103a (one -gencode, translation units compiled
in parallel) and, where torch's headers and a C++ compiler for them are at hand, the Python module
_binding with g++ against the installed torch; liboracle.so is built separately by ``oracle.build``."""
from __future__ import annotations

import concurrent.futures
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvevict.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
           "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def binding_command(out: str):
    """g++ on csrc/binding.cpp."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    torch = list(spec.submodule_search_locations)[0]
    inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"], "-I", inc,
            "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
            os.path.join(CSRC, "binding.cpp"), "-o", out, "-L", lib, "-ltorch_python",
            "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib}"]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    headers.append(os.path.join(ROOT, "include", "kvevict.h"))
    cc = nvcc()
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src] + headers):
            jobs.append([cc, *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("compilation failed: " + " ".join(cmd))

    def binding():
        # built for the Python and torch that are installed, which the stamp names; without one it may be of
        # any others
        stamp, made = os.path.join(BUILD, "binding.txt"), BINDING + f".tmp{os.getpid()}"
        for_ = f"python {sys.version_info[:2]} torch {importlib.metadata.version('torch')}"
        if not _stale(BINDING, [os.path.join(CSRC, "binding.cpp"), headers[-1]]) and os.path.exists(stamp):
            with open(stamp) as f:
                if f.read() == for_:
                    return
        run(binding_command(made))
        if os.path.exists(stamp):
            os.remove(stamp)
        os.replace(made, BINDING)
        with open(stamp, "w") as f:
            f.write(for_)

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        bound = ex.submit(binding)
        list(ex.map(run, jobs))
    if jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    try:
        bound.result()
    except Exception as e:  # the library does without: its calls then take the checks of api.py
        if os.path.exists(BINDING):
            os.remove(BINDING)  # one of other sources, another Python or another torch
        sys.stderr.write(f"_binding is not built, the library is: {e}\n")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
