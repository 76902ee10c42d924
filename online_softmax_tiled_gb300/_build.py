"""Build the in-tree CUDA library ``_lib/libattn_gb300.so`` for sm_103a, and the
Python calls of the cache operators, ``_lib/_cache_calls.so``, on top of it.

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel into
``<repo>/_build/`` and linked into one shared library with a C ABI
(``include/attn.h``). The CUDA runtime is linked statically; the driver's
tensor-map encoder is fetched at run time, so the library loads on machines
without a GPU. Rebuilds happen only when a source or header is newer than the
library. The Python calls need the host compiler and the headers of this Python
and the installed torch; they hold for those alone, so what they were built
against is written beside them and a change of it rebuilds them. The library
needs none of that: it is linked even where the calls cannot be built.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
BUILD_DIR = os.path.join(REPO_DIR, "_build")
LIB_DIR = os.path.join(PKG_DIR, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libattn_gb300.so")
CALLS_PATH = os.path.join(LIB_DIR, "_cache_calls.so")
STAMP_PATH = CALLS_PATH + ".stamp"

SOURCES = ["api.cu", "fwd_simt.cu", "fwd_tc.cu", "fwd_tc64.cu", "bwd_aux.cu", "bwd_simt.cu", "bwd_tc.cu",
           "bwd_dq.cu", "decode.cu", "decode_shared.cu", "api_cache.cu", "rope.cu",
           "key_weights.cu", "evict.cu", "api_paged.cu", "cache_append.cu", "decode_window.cu"]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                           "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                           "-I" + INCLUDE, "-I" + CSRC]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _inputs_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("command failed: " + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return res.stdout + res.stderr


def _calls_commands(obj: str, out: str):
    """The host compiler's commands (compile, link) for the Python calls,
    against the installed torch and this Python."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    libs = os.path.join(root, "lib")
    cxx = shutil.which("g++") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
                "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", sysconfig.get_paths()["include"],
                "-isystem", os.path.join(cuda, "include"),
                "-c", os.path.join(CSRC, "py_cache.cpp"), "-o", obj]
    link = [cxx, "-shared", obj, "-o", out, "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-ltorch",
            "-ltorch_cuda", "-lc10", "-lc10_cuda",
            "-L" + LIB_DIR, "-l:" + os.path.basename(LIB_PATH),
            "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    return compile_, link


def calls_stamp() -> str:
    """What the Python calls hold for: this Python and the installed torch."""
    import torch
    return " ".join([str(sysconfig.get_config_var("SOABI")), torch.__version__,
                     f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                     os.path.dirname(os.path.abspath(torch.__file__))])


def calls_current() -> bool:
    """Whether the built Python calls are for this Python and torch."""
    if not (os.path.exists(CALLS_PATH) and os.path.exists(STAMP_PATH)):
        return False
    try:
        with open(STAMP_PATH) as f:
            return f.read() == calls_stamp()
    except ImportError:
        return False


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library if needed; return its path."""
    newest = _inputs_mtime()

    def fresh(path):
        return not force and os.path.exists(path) and os.path.getmtime(path) >= newest
    lib_fresh, calls_fresh = fresh(LIB_PATH), fresh(CALLS_PATH) and calls_current()
    if lib_fresh and calls_fresh:
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        out = _run([nvcc, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj, out

    def compile_calls():
        tmp = CALLS_PATH + ".tmp"
        compile_, link = _calls_commands(os.path.join(BUILD_DIR, "py_cache.o"), tmp)
        _run(compile_)
        return link, tmp

    with ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        calls = None if calls_fresh else ex.submit(compile_calls)
        if not lib_fresh:
            results = list(ex.map(compile_one, SOURCES))
            if verbose or ptxas_info:
                for (_, out), src in zip(results, SOURCES):
                    if out.strip():
                        print(f"--- {src}\n{out}")
            tmp = LIB_PATH + ".tmp"
            _run([nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *[o for o, _ in results]])
            os.replace(tmp, LIB_PATH)
        if calls is not None:
            link, tmp = calls.result()   # (an error of theirs comes behind the linked library)
            _run(link)
            if os.path.exists(STAMP_PATH):
                os.remove(STAMP_PATH)
            os.replace(tmp, CALLS_PATH)
            with open(STAMP_PATH, "w") as f:
                f.write(calls_stamp())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
