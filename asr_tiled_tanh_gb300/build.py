"""Build librnnt_gb300.so in-tree for sm_103a (nvcc, one -gencode, parallel TUs), and beside it
the binding's helper for lists of tensors (g++, torch's headers)."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(BUILD, "librnnt_gb300.so")
LISTS_SRC = os.path.join(CSRC, "lists.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


_lists_tried = False


def lists_path() -> str:
    """The helper for lists of tensors: built for one version of Python and of torch."""
    import torch
    return os.path.join(BUILD, f"rnnt_lists-{sys.version_info[0]}.{sys.version_info[1]}"
                               f"-{torch.__version__}.so")


def _start_lists(force: bool):
    """The compiler of the helper at work on it; None where it is up to date, or cannot be built
    (ops.py then takes lists apart in Python)."""
    global _lists_tried
    path = lists_path()
    fresh = os.path.exists(path) and os.path.getmtime(path) >= os.path.getmtime(LISTS_SRC)
    if (fresh or _lists_tried) and not force:
        return None
    _lists_tried = True
    import torch
    t = os.path.dirname(torch.__file__)
    lib = os.path.join(t, "lib")
    tmp = path + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(t, "include"),
           "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"), LISTS_SRC, "-o",
           tmp, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    os.makedirs(BUILD, exist_ok=True)
    try:
        return tmp, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        print(f"{LISTS_SRC}: not built ({e})", file=sys.stderr)
        return None


def _finish_lists(job):
    if job is None:
        return
    tmp, p = job
    out, _ = p.communicate()
    if p.returncode == 0:
        os.replace(tmp, lists_path())
    else:
        print(f"{LISTS_SRC}: not built\n{out.decode(errors='replace')}", file=sys.stderr)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link the shared library."""
    lists = _start_lists(force)
    try:
        return _build_library(force, verbose)
    finally:
        _finish_lists(lists)


def _build_library(force, verbose):
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
