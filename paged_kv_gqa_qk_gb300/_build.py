"""Build libpkv.so in-tree with nvcc for sm_103a.

Each .cu file of csrc/ is compiled to an object in parallel, then linked into
paged_kv_gqa_qk_gb300/libpkv.so (CUDA runtime linked statically, so the
library loads wherever the driver is present).  csrc/pkv_torch.cpp, the
binding's short way to the calls that take a few microseconds, becomes a
CPython module for the installed torch; where that does not build, the
binding does without it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
FAST_SRC = os.path.join(CSRC, "pkv_torch.cpp")
FAST = os.path.join(HERE, "_pkv_torch.so")
NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I" + os.path.join(HERE, "..", "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(HERE, "..", "include", "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _fast_command(out: str):
    import torch

    base = os.path.dirname(torch.__file__)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            f'-DPKV_TORCH_VERSION="{torch.__version__}"', "-isystem", os.path.join(base, "include"),
            "-I" + sysconfig.get_paths()["include"], FAST_SRC, "-o", out, "-L" + os.path.join(base, "lib"),
            "-lc10", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath," + os.path.join(base, "lib")]


def _build_fast(verbose: bool) -> None:
    tmp = FAST + f".tmp{os.getpid()}"
    try:
        cmd = _fast_command(tmp)
        r = subprocess.run(cmd, capture_output=True, text=True)
    except (ImportError, OSError) as e:
        sys.stderr.write(f"{os.path.basename(FAST)} not built: {e}\n")
        return
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode == 0:
        os.replace(tmp, FAST)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = _sources()
    headers = [d for d in _deps() if not d.endswith(".cu")]
    objs = []
    jobs = []
    for src in srcs:
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [NVCC, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
            jobs.append(cmd)
    torch = importlib.util.find_spec("torch")  # (another torch installed since: built again)
    fast = force or _stale(FAST, [FAST_SRC] + ([torch.origin] if torch and torch.origin else []))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        if fast:
            fast = ex.submit(_build_fast, verbose)
        if jobs:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
            for cmd, r in zip(jobs, results):
                if verbose or r.returncode != 0:
                    sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
                if r.returncode != 0:
                    raise RuntimeError(f"nvcc failed for {cmd[-3]}")
        if fast:
            fast.result()
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else [])
    print(LIB)
