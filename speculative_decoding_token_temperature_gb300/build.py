"""Build the in-tree C-ABI library `libspecdec.so` with nvcc for sm_103a.

Each .cu translation unit is compiled in parallel to an object, then linked into one
shared library next to this file.  The CUDA runtime is linked statically, so loading
the library (e.g. to list its symbols) does not need a GPU.  The library needs nvcc alone
(`python build.py` in a Python without torch builds just that, for C callers); with torch, the
host compiler builds `_cache_calls.so`, the Python side of the cache calls, beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIB_NAME = "libspecdec.so"
LIB_PATH = PKG / LIB_NAME
CALLS_PATH = PKG / "_cache_calls.so"
BUILD_DIR = PKG / "_build"

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-O3"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libspecdec.so")


def _sources():
    return sorted(CSRC.glob("*.cu"))


def _digest(files, *words) -> str:
    h = hashlib.sha256()
    for p in sorted(files):
        h.update(p.name.encode())
        h.update(p.read_bytes())
    for w in (*words, os.uname().machine):
        h.update(w.encode())
    return h.hexdigest()


def _fingerprint() -> str:
    """Of what the library is made from: the CUDA sources and headers."""
    files = [p for g in ("*.cu", "*.cuh", "*.h") for p in CSRC.glob(g)] + list(INCLUDE.glob("*.h"))
    return _digest(files, " ".join(ARCH_FLAGS + NVCC_FLAGS))


def _calls_fingerprint() -> str:
    import torch
    return _digest([CSRC / "cache_calls.cpp", *INCLUDE.glob("*.h")], torch.__version__, sys.version)


def _current(so: Path, stamp: Path, fingerprint: str) -> bool:
    return so.exists() and stamp.exists() and stamp.read_text() == fingerprint


def _calls_command(out: Path) -> list:
    """The host compiler's command for the Python side of the cache calls (csrc/cache_calls.cpp),
    a CPython module on torch's C++ tensors, linked against the library next to it."""
    import torch
    cuda = Path(_nvcc()).resolve().parents[1]
    root = Path(torch.__file__).resolve().parent
    lib = root / "lib"
    inc = [sysconfig.get_paths()["include"], root / "include", root / "include" / "torch" / "csrc" / "api" / "include",
           cuda / "include", INCLUDE]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             *(f"-I{i}" for i in inc), str(CSRC / "cache_calls.cpp"), "-o", str(out), f"-L{lib}", "-lc10", "-lc10_cuda",
             "-ltorch_cpu", "-ltorch_python", "-ltorch", f"-Wl,-rpath,{lib}"])


def build_library(verbose: bool = False, force: bool = False, extra_flags=None) -> Path:
    """Compile every .cu under csrc/ and link libspecdec.so (skipped when up to date).  Needs no torch."""
    stamp, fp = BUILD_DIR / "stamp", _fingerprint()
    if not force and _current(LIB_PATH, stamp, fp):
        return LIB_PATH
    BUILD_DIR.mkdir(exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH_FLAGS + NVCC_FLAGS + list(extra_flags or []) + [f"-I{INCLUDE}", f"-I{CSRC}"]

    def compile_one(src: Path) -> Path:
        obj = BUILD_DIR / (src.stem + ".o")
        cmd = [nvcc, *flags, "-c", str(src), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB_PATH.with_suffix(".so.tmp")
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", str(tmp), *map(str, objs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    stamp.write_text(fp)
    return LIB_PATH


def _compile_calls() -> Path:
    obj = BUILD_DIR / "cache_calls.o"
    BUILD_DIR.mkdir(exist_ok=True)
    cmd = [c for c in _calls_command(obj) if c != "-shared" and not c.startswith(("-l", "-L", "-Wl"))] + ["-c"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for cache_calls.cpp:\n{r.stderr}")
    return obj


def _link_calls(obj: Path) -> None:
    tmp = CALLS_PATH.with_suffix(".so.tmp")
    cmd = [str(obj) if c == str(CSRC / "cache_calls.cpp") else c for c in _calls_command(tmp)]
    cmd += [f"-L{PKG}", "-lspecdec", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {CALLS_PATH.name} failed:\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(verbose: bool = False, force: bool = False, extra_flags=None) -> Path:
    """The library and the Python side of the cache calls, each skipped when up to date."""
    stamp, fp = BUILD_DIR / "calls_stamp", _calls_fingerprint()
    if not force and _current(CALLS_PATH, stamp, fp):
        return build_library(verbose, force, extra_flags)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_calls)
        build_library(verbose, force, extra_flags)
        _link_calls(obj.result())
    stamp.write_text(fp)
    return LIB_PATH


def ensure_built() -> Path:
    return build()


def ptxas_report() -> str:
    """Register / shared-memory usage of every kernel (nvcc -Xptxas -v)."""
    nvcc = _nvcc()
    out = []
    for src in _sources():
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, "-Xptxas", "-v", f"-I{INCLUDE}", f"-I{CSRC}",
               "-c", str(src), "-o", os.devnull]
        r = subprocess.run(cmd, capture_output=True, text=True)
        out.append(r.stderr)
    return "\n".join(out)


if __name__ == "__main__":
    if "--ptxas" in sys.argv:
        print(ptxas_report())
    else:
        make = build if importlib.util.find_spec("torch") else build_library
        print(make(verbose=True, force="--force" in sys.argv))
