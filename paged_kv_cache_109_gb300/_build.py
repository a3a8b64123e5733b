"""Compile the CUDA library (libpa.so) in-tree for sm_103a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpa.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or install the CUDA toolkit)")


def sources() -> list[str]:
    files = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
             if f.endswith((".cu", ".cuh", ".h"))]
    return files + [os.path.join(INCLUDE, "pa.h")]


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build libpa.so next to this file unless it is up to date: the source files
    compile at the same time, then link.  What that makes on its way is in a
    folder of the call's own, so several processes may build at once."""
    if not force and not stale():
        return LIB
    units = [f for f in sources() if f.endswith(".cu")]
    with tempfile.TemporaryDirectory(prefix=".build-", dir=PKG) as tmp:
        objects = [os.path.join(tmp, os.path.basename(f)[:-3] + ".o") for f in units]
        jobs = []
        for src, obj in zip(units, objects):
            cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, *extra_flags, "-c", "-o", obj, src]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
        outputs = [job.communicate()[1] for job in jobs]
        for job, err in zip(jobs, outputs):
            if job.returncode != 0:
                raise RuntimeError(f"nvcc failed ({job.returncode}):\n{err[-4000:]}")
            if verbose:
                print(err)
        lib = os.path.join(tmp, "libpa.so")
        res = subprocess.run([_nvcc(), *ARCH, "-shared", *extra_flags, "-o", lib, *objects],
                             capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stderr[-4000:]}")
        os.replace(lib, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
