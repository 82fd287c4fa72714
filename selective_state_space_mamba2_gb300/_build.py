"""Builds the CUDA library ``libssd_gb300.so`` in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process (in parallel),
then linked; nothing is installed outside the package directory.  Beside it
the CPython module ``_kv_calls.so`` (host compiler, torch's headers), which
marshals the arguments of the attention-side calls.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libssd_gb300.so")

SOURCES = ["api.cu", "decode.cu", "prefill_simt.cu", "prefill_tc.cu", "prefill_static.cu", "conv1d.cu", "mamba1.cu", "metadata.cpp",
           "kv_api.cu", "kv_tables.cu", "kv_tokens.cu", "kv_attention_simt.cu", "kv_attention_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


CALLS = "kv_calls.cpp"
CALLS_LIB = os.path.join(PKG, "_kv_calls.so")


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _headers_mtime() -> float:
    paths = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, src + ".o")
    srcp = os.path.join(CSRC, src)
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(srcp)
            and os.path.getmtime(obj) >= _headers_mtime() and not verbose_ptxas):
        return obj
    tmp = obj + ".tmp.%d" % os.getpid()  # per process: concurrent builds (one per rank) never share a file
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", srcp, "-o", tmp]
    if src.endswith(".cpp"):
        cmd = [nvcc(), "-x", "c++"] + NVCC_FLAGS + ["-c", srcp, "-o", tmp]
    elif verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, res.stdout, res.stderr))
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    os.replace(tmp, obj)
    return obj


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _calls_key() -> str:
    """What the marshalling module is compiled against besides this repository's sources."""
    import torch
    return "\n".join([torch.__version__, _torch_dir(), "cxx11abi %d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
                      sysconfig.get_config_var("EXT_SUFFIX") or "", sysconfig.get_paths()["include"]])


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _compile_calls() -> str:
    obj, srcp = os.path.join(BUILD, CALLS + ".o"), os.path.join(CSRC, CALLS)
    key, keyp = _calls_key(), os.path.join(BUILD, CALLS + ".key")
    if (os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(srcp), _headers_mtime())
            and _read(keyp) == key):
        return obj
    import torch
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    tmp = obj + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c", srcp, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (CALLS, res.stdout, res.stderr))
    os.replace(tmp, obj)
    with open(tmp, "w") as f:
        f.write(key)
    os.replace(tmp, keyp)
    return obj


def _link_calls(obj: str) -> None:
    if os.path.exists(CALLS_LIB) and os.path.getmtime(CALLS_LIB) >= os.path.getmtime(obj):
        return
    tmp = CALLS_LIB + ".tmp.%d" % os.getpid()
    # torch's libraries are loaded already when the module is; ours is found beside it
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(_torch_dir(), "lib"), "-lc10", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, CALLS_LIB)


def _link(objs) -> None:
    if os.path.exists(LIB) and all(os.path.getmtime(LIB) >= os.path.getmtime(o) for o in objs):
        return
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart", "-lcuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, LIB)


def build(verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
        calls = calls.result()
    _link(objs)
    _link_calls(calls)
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv))
