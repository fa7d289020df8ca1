"""Build libflashoverlap.so in-tree with nvcc for sm_103a, and the operators' argument marshalling beside it.

Every translation unit is compiled in parallel to an object file under
``ag_gemm_gb300/_build/`` and then linked into one shared library with the
CUDA runtime linked statically. Nothing is written outside the package.

The marshalling module needs g++ and torch's headers besides. It only makes
Python's calls of the operators shorter: where it cannot be built, the library
is there all the same, and the binding does its work in Python.
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libflashoverlap.so")

SOURCES = ["fo_plan.cpp", "fo_api.cu", "fo_kern_rs.cu", "fo_kern_dp.cu", "fo_kern_ag.cu", "fo_kern_part.cu",
           "fo_noalloc.cu", "fo_attn.cu", "fo_norm.cu", "fo_quant.cu", "fo_rope.cu", "fo_gemm_fp8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libflashoverlap.so")


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "flashoverlap.h"), __file__]
    return max(os.path.getmtime(p) for p in paths)


def torch_version() -> str:
    """torch's version as it names itself, without importing it; "" where there is none."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return ""
    try:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        found = None
    return found.group(1) if found else "unknown"


def marshal_path() -> str:
    """Where the marshalling module for this interpreter and this torch is: it reads both's objects, so one that was
    built for others is not it."""
    return os.path.join(BUILD, f"_fo_marshal-torch{torch_version()}.{sysconfig.get_config_var('SOABI')}.so")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of libflashoverlap.so."""
    stale = [force or not os.path.exists(f) or os.path.getmtime(f) < _deps_mtime() for f in (LIB, marshal_path())]
    if not any(stale):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                    f"-I{INCLUDE}", f"-I{CSRC}"] + list(extra_flags)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        if verbose:
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal, nvcc) if stale[1] else None
        if stale[0]:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + ".tmp"
            cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
            os.replace(tmp, LIB)
        if marshal is not None:
            try:
                _link_marshal(marshal.result())
            except (RuntimeError, OSError) as e:
                sys.stderr.write(f"the operators' argument marshalling was not built (Python does its work): {e}\n")
                if os.path.exists(marshal_path()):
                    os.remove(marshal_path())   # of older sources
    return LIB


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("torch not found: the argument marshalling module is compiled with its headers")
    return os.path.dirname(spec.origin)


def _cxx(cmd, what: str) -> None:
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found for the argument marshalling module")
    res = subprocess.run([cxx] + cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join([cxx] + cmd)}\n{res.stdout}\n{res.stderr}")


def _compile_marshal(nvcc: str) -> str:
    """The operators' argument marshalling, a CPython module that reads torch's tensors directly."""
    obj, torch_include = os.path.join(BUILD, "fo_marshal.o"), os.path.join(_torch_dir(), "include")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    includes = [torch_include, os.path.join(torch_include, "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], cuda_include, INCLUDE]
    _cxx(["-O2", "-std=c++17", "-fPIC"] + [f"-I{d}" for d in includes] +
         ["-c", os.path.join(CSRC, "fo_marshal.cpp"), "-o", obj], "compiling the argument marshalling")
    return obj


def _link_marshal(obj: str) -> None:
    """Link it to the library beside it and to torch's (loaded with torch, which comes first)."""
    tmp = marshal_path() + ".tmp"
    _cxx(["-shared", obj, "-o", tmp, "-L", BUILD, "-lflashoverlap", "-L", os.path.join(_torch_dir(), "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"], "linking the argument marshalling")
    os.replace(tmp, marshal_path())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
