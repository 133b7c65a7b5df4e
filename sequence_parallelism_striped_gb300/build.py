"""Build libstriped.so in-tree with nvcc for sm_103a (GB300).

Each translation unit is compiled in parallel; the shared library lands in
``sequence_parallelism_striped_gb300/_build/libstriped.so`` (git-ignored).
No CMake, no torch extension machinery: plain nvcc.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libstriped.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "permute.cu", "attn_simt.cu", "attn_fwd_tc.cu", "attn_fwd_pair.cu", "attn_bwd_tc.cu", "attn_bwd_noalloc.cu",
           "norm_rope.cu", "attn_window_fwd.cu", "attn_window_bwd.cu", "attn_decode.cu", "attn_decode_kv4.cu",
           "attn_decode_kv4_tc.cu", "kv4.cu", "kv_evict.cu", "key_weight.cu",
           "host_model.cpp"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _flags(extra=()):
    return ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
            *ARCH, *extra]


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def binding_path() -> str | None:
    """Where the binding (csrc/binding.cpp: some calls from Python in one step) of this torch, interpreter and source lies,
    built or not.  It reads tensors through torch's inlined headers and calls the library through its header's
    signatures, so one of another torch or header has another name; None if there is no torch or no source."""
    try:
        import torch

        h = hashlib.sha256(f"{torch.__version__} {torch.version.git_version} {sysconfig.get_config_var('SOABI')}".encode())
        for p in (os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "striped.h")):
            with open(p, "rb") as f:
                h.update(f.read())
    except (ImportError, AttributeError, OSError):
        return None
    return os.path.join(BUILD, f"striped_binding-{h.hexdigest()[:16]}.so")


def _build_binding(path: str | None):
    """Compile the binding to `path`.  Returns what went wrong, or None: without it the wrappers do the same work, slower."""
    if path is None:
        return "no torch, or no source"
    tmp = path + f".tmp{os.getpid()}"
    try:
        import torch

        root = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-I", INCLUDE, "-I", os.path.join(root, "include"),
               "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
               os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python",
               "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            return res.stderr or f"g++ ended with {res.returncode}"
        os.replace(tmp, path)
    except Exception as e:  # whatever it is, the library does without
        return f"{type(e).__name__}: {e}"
    for name in os.listdir(BUILD):  # of other sources or another torch
        old = os.path.join(BUILD, name)
        if name.startswith("striped_binding") and name.endswith(".so") and old != path:
            try:
                os.remove(old)
            except OSError:
                pass
    return None


def _report(wrong):
    if wrong:
        print(f"binding.cpp not built, calls go through ctypes alone: {wrong[-2000:]}", file=sys.stderr)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every source and link libstriped.so; returns its path.  A library that is up to date stays, and so does
    the binding of this torch; without one it is tried again."""
    binding = binding_path()
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        if binding is None or not os.path.exists(binding):
            _report(_build_binding(binding))
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        extra = ["-Xptxas", "-v"] if ptxas_info and src.endswith(".cu") else []
        cmd = [nvcc, "-c", os.path.join(CSRC, src), "-o", obj, *_flags(extra)]
        if src.endswith(".cpp"):
            cmd = [nvcc, "-x", "c++", "-c", os.path.join(CSRC, src), "-o", obj, "-O2", "-std=c++17",
                   "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            print(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        wrong = ex.submit(_build_binding, binding)
        objs = list(ex.map(compile_one, SOURCES))
        _report(wrong.result())
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", *ARCH, "-o", tmp, *objs, "-lcuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))
