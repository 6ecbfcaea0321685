"""Build libattn.so in-tree with nvcc for sm_103a, and the Python entry of the
decoding-step calls (_binding.so) with the host compiler.

    python -m exact_attention_75_gb300.build [--force]

Each .cu file under csrc/ is compiled in parallel to an object file in
``_build/``, then linked into ``_build/libattn.so`` (CUDA runtime linked
statically; the driver API is reached through cudaGetDriverEntryPointByVersion,
so the library loads on machines without a GPU driver).  A file is recompiled
only when it, or a header under csrc/ or include/, is newer than its object.
csrc/binding.cpp is compiled against the installed torch and Python headers,
again when those change; the library is linked whatever becomes of it, and
without torch it is left out.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libattn.so")
BINDING = os.path.join(BUILD, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                  "-I", CSRC, "-I", INCLUDE, "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn")


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, obj: str, verbose: bool) -> str:
    cmd = [nvcc()] + NVFLAGS + ["-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr[-6000:]}")
    return r.stderr


def _compile_binding(src: str, out: str) -> str:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX", "c++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-Wl,-rpath," + os.path.join(root, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {os.path.basename(src)} failed:\n{r.stderr[-6000:]}")
    os.replace(tmp, out)
    return r.stderr


def _read(path: str) -> Optional[str]:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _torch() -> Optional[str]:
    """What _binding.so is compiled against: Python's ABI, torch's place and
    version.  None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    root = os.path.dirname(spec.origin)
    with open(os.path.join(root, "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{root}\n{f.read()}"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libattn.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr = _newest_header()
    jobs = {}
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr):
            jobs[s] = o
    src = os.path.join(CSRC, "binding.cpp")
    header = os.path.getmtime(os.path.join(INCLUDE, "attn.h"))
    stamp, against = BINDING + ".txt", _torch()
    if against is None:
        sys.stderr.write("torch is not installed: the Python entry of the rotary and paged calls "
                         "(_binding.so) is not built\n")
    bind = against is not None and (
        force or not os.path.exists(BINDING) or _read(stamp) != against or
        os.path.getmtime(BINDING) < max(os.path.getmtime(src), header))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, len(jobs) + bind))) as ex:
        binding = ex.submit(_compile_binding, src, BINDING) if bind else None
        for f in cf.as_completed([ex.submit(_compile, s, o, verbose) for s, o in jobs.items()]):
            log = f.result()
            if verbose and log:
                sys.stderr.write(log)
        if jobs or not os.path.exists(LIB):
            tmp = LIB + ".tmp"
            r = subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs,
                               capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
            os.replace(tmp, LIB)
        if binding is not None:
            binding.result()
            with open(stamp, "w") as f:
                f.write(against)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
