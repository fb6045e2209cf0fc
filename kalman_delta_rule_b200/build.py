"""Build libkdn.so in-tree with nvcc for sm_100a (B200).

Each ``csrc/*.cu`` is compiled to an object in ``_build/`` (in parallel, only when it
or a header changed) and the objects are linked into ``kalman_delta_rule_b200/libkdn.so``.
``csrc/kdn_marshal.cpp`` (the binding's native path from torch tensors to the C ABI; host code only)
becomes the extension module ``_kdn_marshal.so`` beside it, with g++ and torch's headers.  The library needs nvcc
alone; where torch, its headers, Python's or g++ are missing the module is left out with a warning, and
the wrappers do without it.
Usage: ``python -m kalman_delta_rule_b200.build [--force] [--verbose]``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libkdn.so")
MARSHAL = os.path.join(PKG, "_kdn_marshal.so")
OBJ_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3",
                     "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def marshal_abi() -> str:
    """What the extension module is built for (``torch`` importable): torch's version and the interpreter's ABI."""
    import torch
    return f"{torch.__version__} {sys.implementation.cache_tag}"


def marshal_missing() -> str | None:
    """What the extension module cannot be built without and is not here; None if all is."""
    try:
        import torch
    except ImportError:
        return "torch"
    if not os.path.isdir(os.path.join(os.path.dirname(torch.__file__), "include", "torch")):
        return "torch's headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None if shutil.which("g++") else "g++"


def build_marshal(force: bool = False) -> str | None:
    """The binding's extension module (torch's headers and libraries, the running interpreter's ABI); None where something
    that it needs is missing.  Built again when its source, the ABI's header, torch or the interpreter has changed."""
    missing = marshal_missing()
    if missing:
        warnings.warn(f"{os.path.basename(MARSHAL)} is not built: no {missing}; the wrappers take their calls through ctypes")
        return None
    src, record, abi = os.path.join(CSRC, "kdn_marshal.cpp"), os.path.join(OBJ_DIR, "_kdn_marshal.abi"), marshal_abi()
    newest = max(os.path.getmtime(p) for p in (src, __file__, os.path.join(ROOT, "include", "kdn.h")))
    if not force and os.path.exists(MARSHAL) and os.path.getmtime(MARSHAL) >= newest and os.path.exists(record):
        with open(record) as f:
            if f.read() == abi:
                return MARSHAL
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    inc = [os.path.join(ROOT, "include"), os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f'-DKDN_MARSHAL_ABI="{abi}"']
    cmd += ["-I" + i for i in inc] + [src, "-o", tmp, "-L" + os.path.join(home, "lib"), "-Wl,-rpath," + os.path.join(home, "lib")]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{p.stderr}")
    os.replace(tmp, MARSHAL)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(record, "w") as f:
        f.write(abi)
    return MARSHAL


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = max([os.path.getmtime(h) for h in _headers()] + [os.path.getmtime(__file__)])
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_time):
            return obj, None
        cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{p.stderr}")
        return obj, p.stderr

    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        marshal = ex.submit(build_marshal, force)
        results = list(ex.map(compile_one, srcs))
    objs = [o for o, _ in results]
    if verbose:
        for o, log in results:
            if log:
                print(f"== {os.path.basename(o)}\n{log}")
    if force or not os.path.exists(OUT) or any(os.path.getmtime(o) > os.path.getmtime(OUT) for o in objs):
        tmp = OUT + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{p.stderr}")
        os.replace(tmp, OUT)
    marshal.result()                       # (the library does not depend on it)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
                ptxas_info="--ptxas" in sys.argv))
