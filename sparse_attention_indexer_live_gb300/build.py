"""Compile the sm_103a CUDA library in-tree (nvcc, no torch extension machinery).

Output: sparse_attention_indexer_live_gb300/_build/libdsa_select.so, plus the
ptxas resource report (registers, spills, shared memory) next to it; and, where
torch is installed, the module through which cache.py makes its ordinary calls
(calls_path(): host code, for one Python and one torch).  The library needs
nothing of the module, and cache.py makes its calls without it, a few us slower:
where it does not compile, build() warns and goes on.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
SOURCES = [os.path.join(PKG, "csrc", "dsa_select.cu"), os.path.join(PKG, "csrc", "dsa_indexer.cu"),
           os.path.join(PKG, "csrc", "dsa_attention.cu"), os.path.join(PKG, "csrc", "dsa_cache.cu"),
           os.path.join(PKG, "csrc", "dsa_cache_attention.cu"), os.path.join(PKG, "csrc", "dsa_cache_tile.cu")]
HEADERS = [os.path.join(INCLUDE, "dsa_select.h"), os.path.join(PKG, "csrc", "dsa_internal.h"),
           os.path.join(PKG, "csrc", "dsa_cache.h")]
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libdsa_select.so")
CALLS_SOURCE = os.path.join(PKG, "csrc", "cache_calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return found


def calls_path() -> str | None:
    """The module built from cache_calls.cpp (None without torch)."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = ""
    return os.path.join(BUILD_DIR, f"cache_calls.torch{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _older(target, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in sources)


def stale() -> bool:
    return _older(LIB_PATH, SOURCES + HEADERS)


def _build_calls(target, cuda_home) -> None:
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    include = [INCLUDE, os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda_home, "include")]
    tmp = f"{target}.tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{d}" for d in include), "-o", tmp, CALLS_SOURCE,
           "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stderr[-4000:])
    os.replace(tmp, target)


def build(force: bool = False) -> str:
    """Compile every translation unit in parallel, then link the library."""
    from concurrent.futures import ThreadPoolExecutor
    calls = calls_path()
    if calls and not force and not _older(calls, [CALLS_SOURCE, HEADERS[0]]):
        calls = None
    if not calls and not force and not stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = nvcc_path()
    pid = os.getpid()
    with ThreadPoolExecutor(1) as other:
        job = other.submit(_build_calls, calls, os.path.dirname(os.path.dirname(nvcc))) if calls else None
        if force or stale():
            _build_library(nvcc, pid)
        try:
            if job:
                job.result()
        except Exception as e:
            if os.path.exists(calls):  # of older sources
                os.remove(calls)
            warnings.warn(f"cache_calls was not built, the cache's calls take a few us more each: {e}", RuntimeWarning,
                          stacklevel=2)
    return LIB_PATH


def _build_library(nvcc, pid) -> None:
    from concurrent.futures import ThreadPoolExecutor

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + f".{pid}.o")
        cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xptxas", "-v",
               "-Xcompiler", "-fPIC", "-c", "-I", INCLUDE, "-o", obj, src]
        res = subprocess.run(cmd, capture_output=True, text=True)
        return obj, " ".join(cmd) + "\n" + res.stdout + res.stderr, res.returncode

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    with open(os.path.join(BUILD_DIR, "ptxas.txt"), "w") as f:
        f.write("\n".join(log for _, log, _ in results))
    bad = [log for _, log, rc in results if rc != 0]
    if bad:
        raise RuntimeError("nvcc failed:\n" + bad[0][-4000:])
    tmp = LIB_PATH + f".tmp{pid}"
    res = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _, _ in results]],
                         capture_output=True, text=True)
    for o, _, _ in results:
        os.remove(o)
    if res.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + res.stderr[-4000:])
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force=True))
