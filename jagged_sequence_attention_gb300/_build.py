"""In-tree build of libjfa.so for sm_103a (nvcc, no cmake).

Each translation unit compiles in its own process; the objects link into
``jagged_sequence_attention_gb300/libjfa.so`` with the CUDA runtime linked
statically, so the library loads on a machine without a GPU driver (tests that
only need the host planner) and only needs the driver when a CUDA call runs.  The
paged cache's compiled Python calls are built beside it (``_cache_calls`` with the
interpreter's own suffix, host code against torch's headers).  The library needs neither
torch nor Python's headers: where the calls cannot be compiled, build() warns and the
library is complete without them.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libjfa.so")
# compiled Python calls of the paged cache (the suffix names the interpreter and the machine)
CALLS = os.path.join(PKG, "_cache_calls" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "plan.cpp", "fwd.cu", "fwd_short.cu", "fwd_pack.cu", "bwd.cu", "bwd_dq.cu", "bwd_fused.cu", "bwd_short.cu", "f32.cu", "static_scratch.cu",
           "cache.cu", "cache_append.cu", "cache_simt.cu", "cache_decode.cu", "cache_chunk.cu", "cache_split.cu",
           "cache_quant.cu", "cache_decode4.cu", "cache_blocks.cu", "cache_join.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return (["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
            + ARCH + list(extra))


def _digest(extra) -> str:
    h = hashlib.sha256()
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(INCLUDE, "jfa.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(_flags(extra)).encode())
    return h.hexdigest()


def _calls_command(out: str):
    """The compile command of the Python extension (host code only, against torch's headers)."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], INCLUDE, "/usr/local/cuda/include", os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include")]
    return ([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{i}" for i in inc]
            + [os.path.join(CSRC, "cache_calls.cpp"), "-o", out, "-L" + os.path.join(root, "lib"), "-lc10",
               "-lc10_cuda", "-ltorch_python", "-ltorch_cpu", "-ltorch"])


def _build_calls(force: bool):
    """Compile the Python extension if its sources, its command, torch or the interpreter have
    changed.  Returns what went wrong, if anything; there is no extension then, as an older one
    might not fit the library."""
    stamp = os.path.join(BUILD, "cache_calls.stamp")
    tmp = CALLS + f".tmp{os.getpid()}"
    try:
        import torch
        cmd = _calls_command(tmp)
        h = hashlib.sha256(" ".join([*_calls_command(CALLS), torch.__version__, str(torch.version.git_version),
                                     sys.version]).encode())
        for path in (os.path.join(CSRC, "cache_calls.cpp"), os.path.join(INCLUDE, "jfa.h")):
            with open(path, "rb") as f:
                h.update(f.read())
        if not force and os.path.exists(CALLS) and _stamped(stamp, h.hexdigest()):
            return None
        r = subprocess.run(cmd, capture_output=True, text=True)
        error = None if r.returncode == 0 else r.stdout + r.stderr
    except (ImportError, OSError) as e:  # no torch, or no compiler
        error = str(e)
    untagged = os.path.join(PKG, "_cache_calls.so")  # builds once left it under this name
    for old in (untagged, *([CALLS, stamp] if error else [])):
        if os.path.exists(old):
            os.remove(old)
    if error:
        return error
    os.replace(tmp, CALLS)
    with open(stamp, "w") as f:
        f.write(h.hexdigest())
    return None


def _stamped(path: str, digest: str) -> bool:
    if not os.path.exists(path):
        return False
    with open(path) as f:
        return f.read().strip() == digest


def build(force: bool = False, extra_flags=(), verbose: bool = False) -> str:
    """Compile (what has changed) and return the path of libjfa.so."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_build_calls, force)
        _build_library(force, extra_flags, verbose)
        error = calls.result()
    if error:
        warnings.warn("the paged cache's compiled Python calls were not built (jfa.jfa_cache_create will refuse):\n"
                      + error, RuntimeWarning, stacklevel=2)
    return LIB


def _build_library(force: bool, extra_flags, verbose: bool):
    stamp = os.path.join(BUILD, "libjfa.stamp")
    dig = _digest(extra_flags)
    if not force and os.path.exists(LIB) and _stamped(stamp, dig):
        return
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + _flags(extra_flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc, "-x", "c++"] + cmd[1:]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {src}\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for _, err in results:
            if err:
                print(err, file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(dig)


def build_variant(name: str, defines, sources=("fwd.cu",), verbose: bool = False) -> str:
    """A test build of the library: `sources` compiled again with the extra -D `defines`,
    linked with the main build's objects for the other sources, as _build/lib<name>.so.
    Returns its path.  The main library is built first if needed."""
    build()
    out_dir = os.path.join(BUILD, name)
    os.makedirs(out_dir, exist_ok=True)
    lib = os.path.join(BUILD, f"lib{name}.so")
    extra = [f"-D{d}" for d in defines]
    stamp = os.path.join(out_dir, "stamp")
    dig = _digest(extra) + ",".join(sources)
    if os.path.exists(lib) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == dig:
                return lib
    nvcc = _nvcc()
    objs = []
    for src in SOURCES:
        base = os.path.splitext(src)[0] + ".o"
        if src in sources:
            obj = os.path.join(out_dir, base)
            cmd = [nvcc] + _flags(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"compile failed: {src}\n{r.stdout}\n{r.stderr}")
            objs.append(obj)
        else:
            objs.append(os.path.join(BUILD, base))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"], capture_output=True,
                       text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    with open(stamp, "w") as f:
        f.write(dig)
    return lib


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force=True, extra_flags=extra, verbose=v))
