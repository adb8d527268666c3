"""Build libgdn.so in-tree with nvcc for sm_103a (GB300).

Each .cu translation unit compiles in parallel into ``_build/`` at the repo
root; the objects link into ``hybrid_gated_deltanet_gb300/libgdn.so`` with the
CUDA runtime linked statically.  ``gdn_marshal.cpp`` (checks of tensors, against torch's
headers) becomes the extension module ``_marshal.so`` beside it.  Usage: ``python -m hybrid_gated_deltanet_gb300.build``.

libgdn.so needs nvcc alone (``python hybrid_gated_deltanet_gb300/build.py`` where there is no torch): ``_marshal.so`` is left out where
the headers for it are missing, and if its compilation fails, the error comes after libgdn.so is in its place.
"""
from __future__ import annotations

import importlib.util
import os
import platform
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdn.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
STAMP = os.path.join(PKG, "_marshal.stamp")  # the Python and torch that _marshal.so was compiled against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["gdn_api.cu", "gdn_decode.cu", "gdn_prefill.cu", "gdn_chunk16.cu", "gdn_noalloc.cu", "gdn_proj.cu",
           "gdn_attn.cu", "gdn_attn_tree.cu", "gdn_tree.cu", "gdn_tables.cu", "gdn_rope.cu", "gdn_few.cu", "gdn_wide.cu",
           "gdn_lora.cu"]
MARSHAL_SOURCE = "gdn_marshal.cpp"
HEADERS = ["gdn_common.cuh", "gdn_gemm.cuh", "gdn_internal.h", "gdn_prefill_common.cuh", "gdn_tc.cuh", "gdn_tma.cuh"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                   "-I", os.path.join(ROOT, "include")] + list(extra)


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [MARSHAL_SOURCE]] + [os.path.join(ROOT, "include", "gdn.h"),
                                                                   os.path.abspath(__file__)]
    return max(os.path.getmtime(p) for p in paths)


# ELF e_machine of the host, so that a library built on another architecture is never taken as current.
_ELF_MACHINE = {"x86_64": 62, "amd64": 62, "aarch64": 183, "arm64": 183}


def _built_here(path: str) -> bool:
    want = _ELF_MACHINE.get(platform.machine().lower())
    try:
        with open(path, "rb") as f:
            head = f.read(20)
    except OSError:
        return False
    if len(head) < 20 or head[:4] != b"\x7fELF":
        return False
    return want is None or int.from_bytes(head[18:20], "little") == want


def _current(path: str) -> bool:
    return os.path.exists(path) and _built_here(path) and os.path.getmtime(path) >= _newest_input()


def marshal_key() -> str:
    """The Python and torch whose layouts _marshal.so relies on (read without importing torch; "" without one)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return ""
    with open(os.path.join(spec.submodule_search_locations[0], "version.py")) as f:
        version = re.search(r"^__version__\s*(?::[^=]*)?=\s*['\"](.+?)['\"]", f.read(), re.M)
    return f"{sys.implementation.cache_tag} {sysconfig.get_platform()} torch {version.group(1)}"


def marshal_fits() -> bool:
    """_marshal.so is here and was compiled against the Python and torch that are here."""
    try:
        with open(STAMP) as f:
            return os.path.exists(MARSHAL) and f.read() == marshal_key()
    except OSError:
        return False


def _marshal_missing() -> str:
    """What _marshal.so cannot be compiled without and is not here ("" if nothing)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "torch"
    for header in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                   os.path.join(spec.submodule_search_locations[0], "include", "torch", "csrc", "Dtype.h")):
        if not os.path.exists(header):
            return header
    return ""


def _build_marshal():
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    includes = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared"]
    cmd += [f"-I{d}" for d in includes] + [os.path.join(CSRC, MARSHAL_SOURCE), "-o", tmp]
    cmd += ["-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {MARSHAL_SOURCE}:\n{res.stdout}\n{res.stderr}")
    if os.path.exists(STAMP):  # (a stamp never stands beside a module that it is not of)
        os.remove(STAMP)
    os.replace(tmp, MARSHAL)
    with open(STAMP, "w") as f:
        f.write(marshal_key())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libgdn.so and _marshal.so, each unless it exists, was built for this host's
    architecture (_marshal.so: and Python and torch) and is newer than every source, header and this script."""
    marshal, missing = None, ""
    with ThreadPoolExecutor(1) as ex:
        if force or not _current(MARSHAL) or not marshal_fits():
            missing = _marshal_missing()
            if not missing:
                marshal = ex.submit(_build_marshal)
        if force or not _current(LIB):
            _build_lib(verbose, ptxas_info)
        if marshal:
            marshal.result()
    if missing and missing != "torch":
        warnings.warn(f"_marshal.so is not built: {missing} not found; the calls of binding.py on trees and page tables need it")
    return LIB


def _build_lib(verbose: bool, ptxas_info: bool):
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + _flags(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        return obj, res.stderr

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                print(log, file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-cudart", "static"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
