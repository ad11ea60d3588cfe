"""Compile the CUDA sources of this package into libfa.so (sm_103a), in place.

Each translation unit is compiled by its own nvcc process (in parallel), then
the objects are linked into ``libfa.so`` next to this file.  The CUDA runtime
is linked statically, and the driver's tensor-map encoder is looked up at run
time, so the library loads on a machine without a GPU driver (for the
symbol-export tests) and runs on any sm_103 device.
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
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa.so")
# the debug build: kernels with index checks (FA_DEBUG), objects and library of its own
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(HERE, "libfa_debug.so")
SOURCES = ["fa_api.cu", "fwd_tc.cu", "fwd_f32.cu", "bwd_tc.cu", "bwd_aux.cu", "fa_noalloc.cu", "fwd_fp8.cu",
           "ops_api.cu", "qk_norm_rope.cu", "kv4.cu", "kv4_attn_d64.cu", "kv4_attn_d128.cu", "plan.cu"]
HEADERS = ["ptx.cuh", "internal.h", "bwd_sched.cuh", "fp8.h", "tiles.cuh", "fwd_common.cuh",
           "ops.h", "kv4.cuh", "kv4_ring.cuh", "kv4_attn.cuh"]
# the short way from Python to the C entry points (a CPython extension; gcc, torch's headers)
LAUNCH_SOURCE = os.path.join(CSRC, "launch.cpp")
LAUNCH = os.path.join(HERE, "_launch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa.so")


def _deps():
    return ([os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(CSRC, h) for h in HEADERS]
            + [os.path.join(ROOT, "include", "fa.h"), os.path.abspath(__file__)])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, extra: list[str], build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if "-v" in extra and r.stderr:
        print(r.stderr, end="")
    return obj


def linked_against() -> str | None:
    """The Python and the torch that _launch.so is built for, as text; None without torch.
    (Read from torch's files: importing it takes seconds.)"""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    where = list(spec.submodule_search_locations)[0]
    with open(os.path.join(where, "version.py")) as f:
        return "\n".join([str(sysconfig.get_config_var("SOABI")), where, f.read()])


def build_launch(force: bool = False) -> str:
    """Build _launch.so if its source is newer or it was built for another Python or torch
    (or if forced); returns its path."""
    made_for, note = linked_against(), os.path.join(BUILD, "launch_made_for.txt")
    if made_for is None:
        raise RuntimeError("torch is not installed: the operators around the attention need it")
    if not force and os.path.exists(LAUNCH) and os.path.exists(note) and all(
            os.path.getmtime(p) <= os.path.getmtime(LAUNCH) for p in (LAUNCH_SOURCE, os.path.abspath(__file__))):
        with open(note) as f:
            if f.read() == made_for:
                return LAUNCH
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = LAUNCH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", cuda, "-o", tmp, LAUNCH_SOURCE, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on launch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LAUNCH)
    os.makedirs(BUILD, exist_ok=True)
    with open(note, "w") as f:
        f.write(made_for)
    return LAUNCH


def build(force: bool = False, extra_flags: list[str] | None = None, verbose: bool = False,
          debug: bool = False) -> str:
    """Build libfa.so (debug: libfa_debug.so, with the kernels' index checks) if any
    source is newer than it (or if forced), and, with torch installed, _launch.so; returns
    the library's path.  The library is in place also where _launch.so fails to build."""
    lib, build_dir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    with_torch = linked_against() is not None
    if not force and up_to_date(lib):
        if with_torch:
            build_launch()
        return lib
    os.makedirs(build_dir, exist_ok=True)
    extra = list(extra_flags or [])
    if debug:
        extra += ["-DFA_DEBUG"]
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        launch = ex.submit(build_launch, force) if with_torch else None
        objs = list(ex.map(lambda s: _compile(s, extra, build_dir), SOURCES))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if launch is not None:
        launch.result()
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
