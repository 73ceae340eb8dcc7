"""Builds ``libmm.so`` (the C-ABI library of include/mm.h) in-tree for sm_103a.

Each ``csrc/*.cu`` is compiled by nvcc in parallel, then linked with the
static CUDA runtime into ``mixture_experts_layer_mm_gb300/libmm.so``. A file is
recompiled only when it or a header is newer than its object.

``csrc/marshal.cpp``, the binding's argument marshalling as a Python extension
(``_marshal``), is built beside it against the torch that is installed. The
package works without it (``_lib.py`` marshals in Python, more slowly), so where
it cannot be built the build says so, removes an earlier one and goes on.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmm.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL_HEADER = os.path.join(INCLUDE, "mm.h")
# Of this Python version: the extension uses more than its stable ABI.
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmm.so")


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _headers_mtime()):
        return obj
    cmd = [nvcc(), "-c", src, "-o", obj] + NVCC_FLAGS + extra
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def marshal_tag() -> str:
    """What the extension has to be built from: its source, the C ABI, and the
    torch and Python at hand."""
    import torch
    h = hashlib.sha256()
    for path in (MARSHAL_SRC, MARSHAL_HEADER):
        with open(path, "rb") as f:
            h.update(f.read())
    h.update(f"{torch.__version__} {sysconfig.get_config_var('EXT_SUFFIX')}".encode())
    return h.hexdigest()[:16]


def _compile_marshal() -> str | None:
    """The object of marshal.cpp; None (with a line saying why) if it does not compile."""
    try:
        import torch
        tag = marshal_tag()
        obj = os.path.join(BUILD, f"marshal.cpp.{tag}.o")
        if os.path.exists(obj):
            return obj
        inc = os.path.join(os.path.dirname(torch.__file__), "include")
        cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
        cmd = [os.environ.get("CXX", "g++"), "-c", MARSHAL_SRC, "-o", obj + ".tmp", "-O2",
               "-std=c++17", "-fPIC", "-w", f'-DMARSHAL_TAG="{tag}"', "-I" + INCLUDE, "-I" + inc,
               "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
               "-I" + sysconfig.get_paths()["include"], "-I" + cuda_inc]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(((r.stderr or r.stdout).strip().splitlines() or ["compiler failed"])
                               [-1][:200])
        os.replace(obj + ".tmp", obj)
        return obj
    except Exception as e:  # no compiler, no headers: the package works without
        print(f"_marshal not built (calls are marshalled in Python): {e}")
        return None


def _link_marshal(obj: str | None) -> None:
    """The extension from its object; none, and no earlier one, if that fails."""
    stamp = os.path.join(BUILD, "marshal.linked")  # names the object of MARSHAL
    if obj is not None:
        if os.path.exists(MARSHAL) and os.path.exists(stamp):
            with open(stamp) as f:
                same = f.read() == os.path.basename(obj)
            if same and os.path.getmtime(MARSHAL) >= os.path.getmtime(LIB):
                return
        import torch
        lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", MARSHAL + ".tmp", obj, LIB,
               "-L" + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda",
               "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(MARSHAL + ".tmp", MARSHAL)
            with open(stamp, "w") as f:
                f.write(os.path.basename(obj))
            return
        print("_marshal not built (calls are marshalled in Python): "
              + (r.stderr or r.stdout).strip()[-200:])
    if os.path.exists(MARSHAL):
        os.remove(MARSHAL)


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every csrc/*.cu and link libmm.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = list(extra or [])
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        marshal = marshal.result()
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static",
                                                              "-Xlinker", "-soname,libmm.so",
                                                              "-Xlinker", "-z,defs",
                                                              "-lpthread", "-ldl", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of libmm.so failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_marshal(marshal)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
