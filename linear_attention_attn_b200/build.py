"""Build step of the CUDA library: compiles csrc/*.cu for sm_100a into libla_b200.so (in-tree).

Run ``python -m linear_attention_attn_b200.build`` (or call ``build()``).  Each
.cu file is compiled separately (in parallel) and linked with the static CUDA
runtime; no GPU is needed.  The driver API entry point used for TMA
descriptors is resolved at run time, so nothing links against libcuda.

csrc/la_bind.cpp, the module that hands torch tensors to the operators around
the token mixers, is compiled with g++ against torch's and Python's headers.
Where one of these is missing the library is built without it, with a note on
stderr; those operators' Python functions then say so when they are called.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
from importlib.util import find_spec

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libla_b200.so")
BIND_SRC = os.path.join(CSRC, "la_bind.cpp")
BIND = os.path.join(PKG, "_la_bind.so")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newest(paths):
    return max((os.path.getmtime(p) for p in paths), default=0.0)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    hdr = _newest(_headers())
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr):
        return obj
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _torch_dir() -> str:
    return os.path.dirname(find_spec("torch").origin)


def _bind_includes():
    torch_inc = os.path.join(_torch_dir(), "include")
    return [sysconfig.get_paths()["include"], torch_inc, os.path.join(torch_inc, "torch", "csrc", "api", "include"),
            os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]


def _bind_missing() -> str:
    """What the binding module's build lacks here ("": nothing)."""
    if shutil.which("g++") is None:
        return "g++"
    if find_spec("torch") is None:
        return "torch"
    for h in ("Python.h", os.path.join("torch", "csrc", "autograd", "python_variable.h"), "cuda_runtime_api.h"):
        if not any(os.path.exists(os.path.join(d, h)) for d in _bind_includes()):
            return h
    return ""


def _bind_for() -> str:
    """The Python and torch that a binding module built here is for."""
    return "%s torch %s %s" % (sysconfig.get_config_var("SOABI"), importlib.metadata.version("torch"), _torch_dir())


def _compile_bind(force: bool) -> str:
    obj = os.path.join(OBJ, "la_bind.o")
    stamp = os.path.join(OBJ, "la_bind.for")
    newest = max(os.path.getmtime(BIND_SRC), _newest(glob.glob(os.path.join(INCLUDE, "*.h"))))
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == _bind_for():
                return obj
    py_inc, *others = _bind_includes()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-w", "-I" + py_inc, "-I" + INCLUDE]
    for d in others:
        cmd += ["-isystem", d]
    r = subprocess.run(cmd + ["-c", BIND_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (BIND_SRC, r.stdout, r.stderr))
    with open(stamp, "w") as f:
        f.write(_bind_for())
    return obj


def _link_bind(obj: str) -> None:
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libla_b200.so", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, BIND)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if anything changed) and return the path of libla_b200.so."""
    os.makedirs(OBJ, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(OBJ, "*.o")):
            os.remove(o)
    missing = _bind_missing()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        bind = None if missing else ex.submit(_compile_bind, force)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    if missing:
        sys.stderr.write("%s not found: built without _la_bind.so (the operators around the token mixers from Python)\n"
                         % missing)
        return LIB
    obj = bind.result()
    if force or not os.path.exists(BIND) or os.path.getmtime(BIND) < os.path.getmtime(obj):
        _link_bind(obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
