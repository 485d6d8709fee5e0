"""Build librlt.so (sm_103a) in-tree with nvcc, one object per .cu, compiled in parallel, and the binding's
argument marshaller (_marshal, a CPython module in C) with the host compiler where Python's headers are there: the
binding does without it, a few microseconds a call slower."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librlt.so")
MARSHAL = os.path.join(PKG, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))   # this Python's alone
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librlt")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs() -> list[str]:
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h", ".c"))]
    return files + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _python_headers() -> str | None:
    """The folder of this Python's headers, if it has them."""
    include = sysconfig.get_paths()["include"]
    return include if os.path.exists(os.path.join(include, "Python.h")) else None


def _host_cc() -> str | None:
    return shutil.which("gcc") or shutil.which("cc")


def up_to_date() -> bool:
    made = [LIB] + ([MARSHAL] if _python_headers() and _host_cc() else [])
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_marshal() -> str | None:
    """Compile csrc/marshal.c for this Python; None where its headers or a C compiler are missing."""
    include, cc = _python_headers(), _host_cc()
    if include is None or cc is None:
        sys.stderr.write("paged_kv_looped_gb300: no Python headers or no C compiler; calls are marshalled in Python\n")
        return None
    tmp = MARSHAL + f".tmp{os.getpid()}"
    r = subprocess.run([cc, "-O2", "-Wall", "-Wextra", "-fPIC", "-shared", "-I", INCLUDE, "-I", include,
                        os.path.join(CSRC, "marshal.c"), "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling marshal.c failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    untagged = os.path.join(PKG, "_marshal.so")  # one without an ABI tag, which any Python would load
    if untagged != MARSHAL and os.path.exists(untagged):
        os.remove(untagged)
    return MARSHAL


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link librlt.so next to this file."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        r = subprocess.run([*common, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    build_marshal()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources())) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
