"""Builds libbsmm.so in-tree with nvcc for sm_103a, and _tensor_lists.so, the
part of the Python binding that is compiled against torch.

Each translation unit is compiled in parallel into ``_build/`` at the repository
root; the shared library is linked into this package directory.  A unit is
recompiled when it, or any header under ``csrc/`` or ``include/``, is newer
than its object, and the library linked when an object is newer than it.
_tensor_lists.so fits one torch and one Python: it is compiled again when either
is another than the one noted beside the objects.  What is built takes its place
whole, when it is done.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbsmm.so")
LISTS = os.path.join(PKG, "_tensor_lists.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _lists_abi() -> str:
    """What _tensor_lists.so fits."""
    import torch
    return f"torch {torch.__version__}, C++ ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, Python {sysconfig.get_config_var('SOABI')}"


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _run(cmd: list[str]) -> subprocess.CompletedProcess:
    """Runs a compiler; the file after its -o appears when it has succeeded."""
    at = cmd.index("-o") + 1
    out, part = cmd[at], f"{cmd[at]}.{os.getpid()}.part"
    try:
        r = subprocess.run(cmd[:at] + [part] + cmd[at + 1:], capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(part, out)
    finally:
        if os.path.exists(part):
            os.remove(part)
    return r


def _lists_command(src: str) -> list[str]:
    """Compiles and links _tensor_lists.so with the host compiler."""
    import torch
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    base = os.path.dirname(torch.__file__)
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], src, "-o", LISTS,
            "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (as needed) and link libbsmm.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdr_time = _newest_header()
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        stale = force or not os.path.exists(obj) or \
            os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time)
        if stale:
            cmd = [nvcc, *ARCH, *CFLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)
    src = os.path.join(CSRC, "tensor_lists.cpp")
    abi, noted = _lists_abi(), os.path.join(BUILD, "_tensor_lists.abi")
    if force or not os.path.exists(LISTS) or os.path.getmtime(LISTS) < os.path.getmtime(src) or _read(noted) != abi:
        jobs.append(_lists_command(src))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
            results = list(ex.map(_run, jobs))
        for cmd, r in zip(jobs, results):
            if verbose or ptxas_info or r.returncode:
                print(" ".join(cmd))
                print(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed for "
                                   f"{next(a for a in cmd if a.endswith(('.cu', '.cpp')))}")
        if src in jobs[-1]:
            with open(noted, "w") as f:
                f.write(abi)
    # also after a build that compiled units and then failed
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(map(os.path.getmtime, objs)):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
        r = _run(cmd)
        if r.returncode:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
