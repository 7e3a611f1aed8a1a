"""Build libpqkv.so (sm_100a) in-tree with nvcc.

    python -m paged_quantized_kv_cache_b200.build [--force] [--verbose]

Every .cu / .cpp under csrc/ is compiled to an object in _build/ (in parallel)
and linked into paged_quantized_kv_cache_b200/libpqkv.so with the static CUDA
runtime; csrc/python/binding.cpp (the Python binding's argument marshalling)
becomes paged_quantized_kv_cache_b200/_binding.so with the host compiler. No GPU
is needed to build.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libpqkv.so")
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_target() -> str:
    """What a build of the Python module is good for: the running Python and torch, whose headers it is compiled
    against. The module holds this as BUILT_FOR."""
    import torch
    return "for python %d.%d, torch %s" % (*sys.version_info[:2], torch.__version__)


def _binding_fits() -> bool:
    with open(BINDING, "rb") as f:
        return binding_target().encode() + b"\0" in f.read()


def _binding_stale() -> bool:
    return _stale(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "pqkv.h"), __file__]) or not _binding_fits()


def _binding_command(out: str):
    """Host compile of the Python module against the headers and libraries of the running Python and torch (which
    its process has loaded before it)."""
    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = ["-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    include = [sysconfig.get_paths()["include"], base, os.path.join(base, "torch", "csrc", "api", "include"),
               os.path.join(ROOT, "include")]
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi())
    return [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", abi,
            "-DPQKV_BUILT_FOR=\"%s\"" % binding_target(),
            *("-isystem" + i for i in include), BINDING_SRC, "-o", out, *libs]


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I" + os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([nvcc] + flags + ["-c", src, "-o", obj])

    binding_tmp = BINDING + ".tmp%d" % os.getpid()
    make_binding = force or _binding_stale()
    if make_binding:
        jobs.append(_binding_command(binding_tmp))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                failed.append(next(a for a in cmd if a.startswith(CSRC)))
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(failed))
    if make_binding:
        os.replace(binding_tmp, BINDING)
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
