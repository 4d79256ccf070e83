"""Build libmoe_route.so in-tree with nvcc for sm_103a, and _block_calls.so.

Each CUDA translation unit is compiled in parallel into ``_build/`` and the
objects are linked into ``padded_permute_combine_gb300/libmoe_route.so``.
``_block_calls.so``, the marshalling of the block operators' calls, is
compiled beside them against the headers of the installed torch.
Run ``python -m padded_permute_combine_gb300.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_route.so")
CALLS_SOURCE = os.path.join(CSRC, "block_calls.cpp")
CALLS = os.path.join(PKG, "_block_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def source_digest() -> str:
    """Hash of every source and header the library is built from."""
    h = hashlib.sha256()
    files = sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                               + glob.glob(os.path.join(INCLUDE, "*.h")))
    for f in files:
        h.update(os.path.basename(f).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS[:-4]).encode())
    return h.hexdigest()[:16]


def _code_only(text: str) -> str:
    """C/C++ source with comments removed and whitespace runs collapsed
    (string and character literals kept as they are)."""
    out, i, n = [], 0, len(text)
    while i < n:
        c = text[i]
        if text.startswith("//", i):
            j = text.find("\n", i)
            i = n if j < 0 else j
        elif text.startswith("/*", i):
            j = text.find("*/", i + 2)
            i = n if j < 0 else j + 2
            out.append(" ")
        elif c in "\"'":
            j = i + 1
            while j < n and text[j] != c:
                j += 2 if text[j] == "\\" else 1
            out.append(text[i:j + 1])
            i = j + 1
        else:
            out.append(c)
            i += 1
    return " ".join("".join(out).split())


def kernel_digest(unit: str) -> str:
    """Hash of one kernel family's translation unit (``csrc/<unit>.cu``), the
    shared headers (every ``.cuh``, and the ``.h`` of ``csrc/`` that the unit
    includes) and the compile flags, comments and layout left out: it
    changes only when what that kernel is compiled from changes, so a profile
    taken on it stays valid while other kernels, or comments, are edited."""
    h = hashlib.sha256()
    files, at = [os.path.join(CSRC, unit + ".cu")], 0
    while at < len(files):  # csrc's .h files that the unit includes, by itself or through one of them
        with open(files[at], encoding="utf-8") as fh:
            own = [os.path.join(CSRC, name) for name in re.findall(r'^#include "(\w+\.h)"', fh.read(), re.M)]
        files += [f for f in own if os.path.exists(f) and f not in files]
        at += 1
    files += sorted(glob.glob(os.path.join(CSRC, "*.cuh")))
    for f in files:
        h.update(os.path.basename(f).encode())
        with open(f, encoding="utf-8") as fh:
            h.update(_code_only(fh.read()).encode())
    h.update(" ".join(ARCH + NVCC_FLAGS[:-4]).encode())
    return h.hexdigest()[:16]


def _compile(src: str, extra: list[str]) -> tuple[str, str]:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
    return obj, res.stderr


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        raise RuntimeError("torch is not installed")
    return os.path.dirname(spec.origin)


def _calls_digest() -> str:
    h = hashlib.sha256()
    for f in [CALLS_SOURCE, os.path.join(_torch_dir(), "version.py")] + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))):
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def _compile_calls() -> str:
    obj = os.path.join(BUILD_DIR, "block_calls.o")
    torch_include = os.path.join(_torch_dir(), "include")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", torch_include, "-isystem",
           os.path.join(torch_include, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", cuda_include, "-c", CALLS_SOURCE, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("%s failed:\n%s" % (" ".join(cmd), res.stderr))
    return obj


def _link_calls(obj: str) -> None:
    """Linked to the libraries by the names under which torch and the loader have them in the process already."""
    tmp = CALLS + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", PKG, "-l:libmoe_route.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, CALLS)
    with open(CALLS + ".digest", "w") as f:
        f.write(_calls_digest() + "\n")


def _fresh(path: str, digest: str) -> bool:
    stamp = path + ".digest"
    return os.path.exists(path) and os.path.exists(stamp) and open(stamp).read().strip() == digest


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every .cu under csrc/ and link the shared library, and the
    module of the block operators' calls. Each is skipped when it was built
    from the current sources (same digest)."""
    again = force or verbose_ptxas
    lib, calls = again or not _fresh(LIB, source_digest()), again or not _fresh(CALLS, _calls_digest())
    if lib or calls:
        os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_calls) if calls else None
        if lib:
            _build_lib(verbose_ptxas)
        if obj is not None:
            _link_calls(obj.result())
    return LIB


def _build_lib(verbose_ptxas: bool) -> None:
    srcs, digest = sources(), source_digest()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(lambda s: _compile(s, extra), srcs))
    for _, err in results:
        if err.strip():
            sys.stderr.write(err)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, LIB)
    with open(LIB + ".digest", "w") as f:
        f.write(digest + "\n")


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
