"""Build libgrok_attn.so (the C-ABI library) in-tree for sm_103a with nvcc, and _binding (a Python extension), the
binding's checks of the calls over parts of a cache, with the host compiler. The extension needs Python's C headers; where there
are none the library is built without it, and sparse.py makes the checks.

Each .cu file is compiled in parallel, then linked into one shared library
next to this file. The CUDA runtime is linked statically; the driver's
tensor-map encoder is looked up at run time, so no libcuda link is needed.
"""
from __future__ import annotations

import concurrent.futures
import os
import platform
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build", platform.machine())
LIB = os.path.join(PKG, "libgrok_attn.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))  # (of this interpreter alone)
SOURCES = ["abi.cu", "rope_append.cu", "prefill.cu", "decode.cu", "selftest.cu", "pipe.cu", "qkv.cu", "slots.cu", "int8_small.cu",
           "kv8_append.cu", "kv8_decode.cu", "kv8_prefill.cu", "kv8_evict.cu",
           "kv_bounds.cu", "block_decode.cu", "shared_prefix.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _stamp_path() -> str:
    return os.path.join(BUILD, "lib.stamp")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "grok_attn.h"))
    files.append(os.path.abspath(__file__))
    return files


def _python_headers() -> str | None:
    """The folder of Python.h, if it is installed."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def up_to_date() -> bool:
    made = [LIB] + ([BINDING] if _python_headers() else [])
    if not all(os.path.exists(p) for p in [*made, _stamp_path()]):
        return False
    with open(_stamp_path()) as f:
        if f.read().strip() != platform.machine():
            return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *CFLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    def compile_binding() -> None:
        headers = _python_headers()
        if headers is None:  # (an older one may not fit the library any more)
            if os.path.exists(BINDING):
                os.remove(BINDING)
            return
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", headers,
               os.path.join(CSRC, "binding.cpp"), "-o", BINDING + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
        os.replace(BINDING + ".tmp", BINDING)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        results = list(ex.map(compile_one, SOURCES))
        binding.result()
    log = "".join(msg for _, msg in results)
    if verbose or ptxas_info:
        print(log)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if os.path.exists(BINDING):
        os.utime(BINDING)  # (as new as the library: what is built together is up to date together)
    with open(_stamp_path(), "w") as f:
        f.write(platform.machine())
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write(log)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))
