"""Build the CUDA library ``libpkv.so`` and the module ``_torch_calls`` in-tree.

Each ``csrc/*.cu`` translation unit is compiled by nvcc for sm_103a in parallel,
then linked into one shared library next to this file.  The CUDA runtime is
linked statically, so loading the library needs only the NVIDIA driver.
``csrc/torch_calls.cpp`` becomes a Python module that links to that library and
to the installed torch, and is built again for another torch or Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build", "pkv")
LIB = os.path.join(HERE, "libpkv.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS = os.path.join(HERE, "_torch_calls.so")
CALLS_TAG = os.path.join(BUILD, "torch_calls.tag")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newest(paths) -> float:
    return max(os.path.getmtime(p) for p in paths)


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "pkv.h")]


def library_up_to_date() -> bool:
    return os.path.exists(LIB) and _newest(_sources() + _headers()) <= os.path.getmtime(LIB)


def _calls_tag() -> str:
    """What _torch_calls.so is built against; it runs with nothing else."""
    import torch
    return f"torch {torch.__version__} python {sys.version_info[0]}.{sys.version_info[1]} {platform.machine()}"


def calls_up_to_date() -> bool:
    if not os.path.exists(CALLS) or not os.path.exists(CALLS_TAG):
        return False
    with open(CALLS_TAG) as f:
        if f.read() != _calls_tag():
            return False
    return _newest([CALLS_SRC, os.path.join(ROOT, "include", "pkv.h")]) <= os.path.getmtime(CALLS)


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r


def _compile_calls(nvcc: str, obj: str) -> None:
    import torch
    torch_root = os.path.dirname(torch.__file__)
    inc = [os.path.join(torch_root, "include"), os.path.join(torch_root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f"-I{os.path.join(ROOT, 'include')}", *[a for p in inc for a in ("-isystem", p)], "-c", CALLS_SRC, "-o", obj],
         f"g++ failed for {CALLS_SRC}")


def _link_calls(obj: str) -> None:
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libpkv.so", "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}",
          "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{torch_lib}"],
         "link failed")
    os.replace(tmp, CALLS)
    with open(CALLS_TAG, "w") as f:
        f.write(_calls_tag())


def _build_library(nvcc: str, ex, verbose: bool, extra_flags) -> None:
    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        r = _run([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj], f"nvcc failed for {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], "link failed")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is out of date of libpkv.so and _torch_calls.so; returns the path of the
    former.  libpkv.so needs nvcc only and is in place before anything about torch can raise."""
    library, calls = force or not library_up_to_date(), True
    try:
        calls = force or not calls_up_to_date()
    except ImportError:  # raised again below, behind the library
        pass
    if not library and not calls:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    calls_obj = os.path.join(BUILD, "torch_calls.o")
    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        compiled = ex.submit(_compile_calls, nvcc, calls_obj) if calls else None
        if library:
            _build_library(nvcc, ex, verbose, extra_flags)
        if compiled is not None:
            compiled.result()
            _link_calls(calls_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
