"""Build libmk.so in-tree with nvcc for sm_100a (no JIT, no torch in it), and _call.so,
the compiled part of the Python binding, with g++ against torch's headers (left out where
torch is not installed: the library does not need it).

``python -m persistent_megakernel_interpreter_b200.build`` or ``build_library()``.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmk.so")
SOURCES = ["api.cu", "megakernel.cu", "megakernel_trace.cu", "baseline.cu", "noalloc.cu", "select.cu", "beam.cu",
           "reorder.cu", "qcache.cu", "pack.cpp", "schedule.cpp"]
HEADERS = ["mk_internal.h", "mk_device.cuh", "pack.h", "qcache.h"]
CALL = os.path.join(PKG, "_call.so")
CALL_STAMP = os.path.join(PKG, "_call.stamp")   # what _call.so was built against
CALL_SOURCE = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None else None


def _call_stamp(torch: str) -> str:
    """The Python and the torch that the binding's machine code belongs to."""
    with open(os.path.join(torch, "version.py")) as f:
        return sys.version + "\n" + f.read()


def _call_stale() -> bool:
    torch = _torch_dir()
    if not os.path.exists(CALL) or not os.path.exists(CALL_STAMP):
        return True
    if torch is not None:
        with open(CALL_STAMP) as f:
            if f.read() != _call_stamp(torch):
                return True
    t = os.path.getmtime(CALL)
    return any(os.path.getmtime(d) > t for d in (CALL_SOURCE, os.path.join(INCLUDE, "mk.h"), os.path.abspath(__file__)))


def _build_call(verbose: bool) -> None:
    """Compile the binding against torch's headers; it links to libmk.so beside it."""
    torch = _torch_dir()
    if torch is None:
        print("torch is not installed: _call.so, the compiled part of the Python binding, is not built", file=sys.stderr)
        return
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    tmp = f"{CALL}.tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{INCLUDE}",
           f"-I{os.path.join(torch, 'include')}", f"-I{os.path.join(torch, 'include', 'torch', 'csrc', 'api', 'include')}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}", CALL_SOURCE, "-o", tmp, f"-L{PKG}", "-l:libmk.so",
           "-Wl,-rpath,$ORIGIN", f"-L{os.path.join(torch, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        subprocess.check_call(cmd)
        os.replace(tmp, CALL)
        with open(CALL_STAMP, "w") as f:
            f.write(_call_stamp(torch))
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "mk.h"),
                                                                 os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every source to an object in parallel, then link libmk.so; then the binding."""
    if not force and not _stale():
        if _call_stale():
            _build_call(verbose)
        return LIB
    tag = f".tmp{os.getpid()}"
    common = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"] + list(extra or [])
    if verbose:
        common.insert(1, "-Xptxas=-v")
    objs = [os.path.join(CSRC, f + tag + ".o") for f in SOURCES]

    def compile_one(i: int) -> None:
        cmd = common + ["-c", "-o", objs[i], os.path.join(CSRC, SOURCES[i])]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.check_call(cmd)

    try:
        with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
            list(ex.map(compile_one, range(len(SOURCES))))
        subprocess.check_call([_nvcc(), *ARCH, "-shared", "-o", LIB + tag] + objs)
        os.replace(LIB + tag, LIB)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    if force or _call_stale():
        _build_call(verbose)
    return LIB


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
