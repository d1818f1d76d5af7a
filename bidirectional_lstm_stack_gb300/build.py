"""Builds liblstmstack.so in-tree from csrc/*.cu for sm_103a, and the Python
module _native.so from csrc/*.cpp.

Each translation unit compiles in parallel with nvcc into ``_build/`` at the
repository root; both are linked next to this file.  No cmake, no torch
extension machinery: the library has a plain C ABI and needs CUDA alone.  The
module takes torch tensors and is linked to the installed torch; without a
torch for CUDA or without Python's headers the library is built all the same,
and a warning says what the module lacks.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblstmstack.so")
NATIVE = os.path.join(PKG, "_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _torch() -> str | None:
    """Folder of the installed torch (found, not imported)."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _module_lacks() -> str | None:
    """What the module cannot be built without and is not there."""
    torch = _torch()
    if torch is None:
        return "torch is not installed"
    if not os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")):
        return f"the torch in {torch} is one without CUDA"
    python = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")):
        return f"there is no Python.h in {python}"
    return None


def _torch_flags():
    torch = _torch()
    home = os.path.dirname(os.path.dirname(_nvcc()))
    paths = [os.path.join(torch, "include"), os.path.join(home, "include"),
             sysconfig.get_paths()["include"]]
    return [f for path in paths for f in ("-isystem", path)]


def sources(ending: str = ".cu"):
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(ending))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    newest_header = max(os.path.getmtime(h) for h in _headers())

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    def objects(srcs, flags, newest):
        """Their objects, and the commands that make those that are missing or old."""
        objs, jobs = [], []
        for src in srcs:
            obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
            objs.append(obj)
            if (force or not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(src)
                    or os.path.getmtime(obj) < newest):
                jobs.append([nvcc, *ARCH, *FLAGS, *flags, *(extra or []), "-c", src, "-o", obj])
        return objs, jobs

    def link(out, runs, args):
        for log in [r.result() for r in runs]:
            if verbose and log:
                print(log)
        if force or runs or not os.path.exists(out):
            tmp = out + f".{os.getpid()}.tmp"
            run([nvcc, *ARCH, "-shared", "-o", tmp, *args])
            os.replace(tmp, out)

    objs, jobs = objects(sources(), [], newest_header)
    lacks = _module_lacks()
    native, native_jobs = [], []
    if not lacks:
        # (another torch is another set of headers)
        newest_torch = os.path.getmtime(os.path.join(_torch(), "version.py"))
        native, native_jobs = objects(sources(".cpp"), _torch_flags(),
                                      max(newest_header, newest_torch))
    with cf.ThreadPoolExecutor(max_workers=max(1, len(jobs) + len(native_jobs))) as ex:
        runs = [ex.submit(run, job) for job in jobs]
        native_runs = [ex.submit(run, job) for job in native_jobs]
        # the library first: it does not depend on the module
        link(LIB, runs, objs)
        if not lacks:
            # (torch's libraries are loaded before the module is)
            link(NATIVE, native_runs,
                 [*native, "-L", PKG, "-llstmstack", "-Xlinker", "-rpath,$ORIGIN", "-L",
                  os.path.join(_torch(), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
                  "-lc10", "-lc10_cuda"])
    if lacks:
        warnings.warn(f"{LIB} is built, {os.path.basename(NATIVE)} (calls on torch tensors) is not: "
                      f"{lacks}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
