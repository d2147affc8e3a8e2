"""Builds the in-tree CUDA library libbdfp4.so for B200 (sm_100a) with nvcc.

Each translation unit compiles to an object of its own, in parallel (one nvcc
process per .cu file, under _build/ beside this file), and nvcc links them
into the shared library.  The Python side of the 8-bit cache's calls
(csrc/py_bdfp8.cpp, an extension module against this interpreter and torch)
compiles beside them and links to that library; where its compiler or headers
are missing the library is built all the same, with a warning."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbdfp4.so")
PY_SRC = os.path.join(CSRC, "py_bdfp8.cpp")
PY_LIB = os.path.join(HERE, "_bdfp8_py.so")
OBJ = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(HERE, "..", "include", "*.h"))


def _stale(target: str, deps: list[str]) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in deps)


def _compile_py(verbose: bool) -> tuple[str, str]:
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(OBJ, "py_bdfp8.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", "-o", obj, PY_SRC,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{d}" for d in (os.path.join(root, "include"), sysconfig.get_paths()["include"],
                                os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"))]]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on py_bdfp8.cpp:\n{r.stdout}{r.stderr}")
    return obj, r.stdout + r.stderr


def _link_py(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.run(["g++", "-shared", "-o", PY_LIB + ".tmp", obj, LIB, "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-ltorch_python",
                    "-ltorch_cpu", "-lc10_cuda", "-lc10"], check=True)
    os.replace(PY_LIB + ".tmp", PY_LIB)


def _build_py(compiled: concurrent.futures.Future, verbose: bool) -> None:
    """The extension module, once the library stands."""
    try:
        obj, log = compiled.result()
        if verbose and log.strip():
            print(log, end="", flush=True)
        _link_py(obj)
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        if os.path.exists(PY_LIB):
            os.remove(PY_LIB)   # of older sources: its calls need not be this library's
        warnings.warn(f"the 8-bit cache's Python calls are not built: {e}", RuntimeWarning, stacklevel=3)


def _compile(src: str, extra: list[str], verbose: bool) -> tuple[str, str]:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *FLAGS, *extra, "-c", "-o", obj, src]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}{r.stderr}")
    return obj, r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, out: str | None = None) -> str:
    """Compile csrc/*.cu into libbdfp4.so (or `out`; then without the extension module) unless it is up to date."""
    target = out or LIB
    headers = _headers()
    lib = force or out is not None or _stale(LIB, [*sources(), *headers])
    py = out is None and (force or _stale(PY_LIB, [PY_SRC, *headers]))
    if not lib and not py:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources() if lib else []
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + py, os.cpu_count() or 1))) as ex:
        ext = ex.submit(_compile_py, verbose) if py else None
        results = list(ex.map(lambda s: _compile(s, extra or [], verbose), srcs))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log, end="", flush=True)
    if lib:
        soname = ["-Xlinker", "-soname=" + os.path.basename(LIB)]   # what the extension module looks for beside it
        cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *soname, "-o", target + ".tmp", *[o for o, _ in results]]
        subprocess.run(cmd, check=True)
        os.replace(target + ".tmp", target)
    if ext is not None:
        _build_py(ext, verbose)
    return target


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None)
