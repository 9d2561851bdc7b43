"""Build liborthrus.so (sm_100a, nvcc) and the native part of its Python binding (g++) in-tree.

    python -m shared_kv_draft_b200.build [--force]
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "liborthrus.so")
OBJ_DIR = os.path.join(HERE, "_build")  # object files, one per translation unit
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SRC = os.path.join(SRC_DIR, "binding.cpp")
BINDING_TAG = os.path.join(OBJ_DIR, "binding.tag")  # the torch and Python it was compiled for
UNITS = [os.path.join(SRC_DIR, u) for u in ("orthrus.cu", "operators.cu")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    out = [os.path.join(INCLUDE, "orthrus.h")]
    for f in sorted(os.listdir(SRC_DIR)):
        if f.endswith((".cu", ".cuh", ".h", ".cpp")):
            out.append(os.path.join(SRC_DIR, f))
    return out


def _newer(path: str, than) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(s) <= os.path.getmtime(path) for s in than)


def library_up_to_date() -> bool:
    return _newer(LIB, [s for s in sources() if s != BINDING_SRC])


def _binding_tag() -> str:
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_up_to_date() -> bool:
    if not _newer(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "orthrus.h")]) or not os.path.exists(BINDING_TAG):
        return False
    with open(BINDING_TAG) as f:
        return f.read() == _binding_tag()


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _includes(path: str, seen: set) -> set:
    """`path` and the project files it includes, directly or not."""
    if path in seen:
        return seen
    seen.add(path)
    with open(path) as f:
        for name in re.findall(r'^\s*#include "([^"]+)"', f.read(), flags=re.M):
            for d in (SRC_DIR, INCLUDE):
                if os.path.exists(os.path.join(d, name)):
                    _includes(os.path.join(d, name), seen)
    return seen


def _run(cmd, verbose):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(os.path.basename(cmd[0]) + " failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    if verbose:
        sys.stderr.write(r.stderr)


def _compile(src: str, force: bool, verbose: bool) -> str:
    """Object file of one translation unit; compiled when one of its files is newer."""
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    if not force and os.path.exists(obj) and all(os.path.getmtime(f) <= os.path.getmtime(obj)
                                                 for f in _includes(src, set())):
        return obj
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "-Xcompiler", "-fPIC", "-I", INCLUDE, "-c", "-o", obj + ".tmp", src]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    _run(cmd, verbose)
    os.replace(obj + ".tmp", obj)
    return obj


def _build_binding(verbose: bool) -> None:
    """Python module over torch's headers, linked with liborthrus.so beside it."""
    import torch
    tag = _binding_tag()
    if os.path.exists(BINDING):  # an old one does not outlive a failure
        os.remove(BINDING)
    root = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda", "include"), sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f'-DORTHRUS_BUILT_FOR="{tag}"']
         + [x for d in inc for x in ("-I", d)] + [BINDING_SRC, "-o", BINDING + ".tmp", "-L", HERE, "-l:liborthrus.so",
                                                  "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"), "-ltorch_python",
                                                  "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"], verbose)
    os.replace(BINDING + ".tmp", BINDING)
    with open(BINDING_TAG, "w") as f:
        f.write(tag)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date. The library needs nvcc alone; where the binding cannot be compiled (no Python headers,
    say), that is a warning, and the tree and rotary calls from Python, which go through it, refuse to run."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    if force or not library_up_to_date():
        with ThreadPoolExecutor(len(UNITS)) as pool:
            objs = list(pool.map(lambda u: _compile(u, force, verbose), UNITS))
        _run([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC", "-o", LIB + ".tmp"]
             + objs, verbose)
        os.replace(LIB + ".tmp", LIB)
    try:
        if force or not binding_up_to_date():
            _build_binding(verbose)
    except (RuntimeError, OSError, ImportError) as e:  # ImportError: no torch
        warnings.warn(f"liborthrus.so is built, its native binding is not: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
