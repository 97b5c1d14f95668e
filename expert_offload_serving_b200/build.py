"""Build libmoe.so in-tree for sm_100a with nvcc.

Every .cu / .cpp under csrc/ is compiled to an object in _build/ (parallel,
skipped when up to date) and linked into expert_offload_serving_b200/libmoe.so;
native.cpp becomes the Python extension _native.so beside it (against torch's
headers and libmoe.so).
Run:  python -m expert_offload_serving_b200.build [--debug] [-v]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe.so")
NATIVE_SRC = os.path.join(PKG, "native.cpp")
NATIVE = os.path.join(PKG, "_native.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include")]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe")


def gxx_path() -> str:
    for cand in (os.environ.get("CXX"), shutil.which("g++")):
        if cand and shutil.which(cand):
            return cand
    raise RuntimeError("g++ not found: the host compiler is required to build libmoe")


def cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp", ".cc")))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "moe.h"))
    return hs


def _compile(src, debug, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest_dep = max(os.path.getmtime(p) for p in [src] + _headers())
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj, ""
    if src.endswith(".cc"):
        # host-only code that uses CPU vector intrinsics: the host compiler
        cmd = [gxx_path(), "-O3", "-std=c++17", "-fPIC", "-pthread", "-Wall", "-I" + os.path.join(ROOT, "include"),
               "-I" + cuda_include(), "-c", src, "-o", obj]
    else:
        cmd = [nvcc_path()] + ARCH + COMMON + ["-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd += ["-x", "cu"]
    if debug:
        cmd += ["-DMOE_DEBUG=1"]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_native() -> str:
    """native.cpp -> an object; the link follows libmoe's."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "native.cpp.o")
    deps = [NATIVE_SRC, os.path.join(ROOT, "include", "moe.h"), torch.__file__]
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(p) for p in deps):
        return obj
    cmd = [gxx_path(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + cuda_include(),
           "-I" + sysconfig.get_paths()["include"], *["-isystem" + p for p in include_paths()], "-c", NATIVE_SRC,
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on native.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_native(obj: str):
    import torch
    if os.path.exists(NATIVE) and os.path.getmtime(NATIVE) >= max(os.path.getmtime(obj), os.path.getmtime(LIB)):
        return
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [gxx_path(), "-shared", "-o", NATIVE, obj, "-L" + PKG, "-l:libmoe.so", "-Wl,-rpath,$ORIGIN", "-L" + tlib,
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _native.so failed:\n{r.stdout}\n{r.stderr}")


def build(debug: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        native = ex.submit(_compile_native)
        results = list(ex.map(lambda s: _compile(s, debug, verbose), srcs))
        native = native.result()
    objs = [o for o, _ in results]
    if verbose:
        for (o, log) in results:
            if log:
                print(f"== {os.path.basename(o)}\n{log}")
    if os.path.exists(LIB) and os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs):
        _link_native(native)
        return LIB
    cmd = [nvcc_path()] + ARCH + ["-shared", "-o", LIB] + objs + ["-Xcompiler", "-fPIC", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _link_native(native)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--debug", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(debug=a.debug, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
