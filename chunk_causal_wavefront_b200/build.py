"""Build libwf.so in-tree with nvcc for sm_100a, and the row operators' torch binding
(_rows_bind.so) with the host compiler.

Usage: python chunk_causal_wavefront_b200/build.py [--force] [--verbose] [--ptxas-info]
(run by path, so that a stale libwf.so is not loaded through the package)
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwf.so")

BIND_SRC = os.path.join(PKG, "bind", "rows_bind.cpp")
# Its name carries the interpreter's ABI, so that no other Python tries to load it.
BIND = os.path.join(PKG, "_rows_bind" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libwf needs the CUDA toolkit to build")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest_dep = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep and not extra:
        return obj
    cmd = [nvcc()] + ARCH + FLAGS + list(extra) + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def torch_version(torch_dir: str) -> str:
    """__version__ of the torch in this directory, without importing it."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return re.search(r"^__version__ = '([^']+)'", f.read(), re.M).group(1)


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """The compiled common case of the row operators' torch-facing calls, against the installed
    torch's headers (found without importing it). It is rebuilt for another torch, whose version it
    carries: the package loads it only under that one."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("torch is not installed")
    torch = os.path.dirname(spec.origin)
    version = torch_version(torch)
    stamp = os.path.join(BUILD, os.path.basename(BIND) + ".torch")
    deps = [BIND_SRC, os.path.join(INCLUDE, "wf.h")]
    if not force and os.path.exists(BIND) and os.path.getmtime(BIND) >= max(map(os.path.getmtime, deps)):
        if os.path.exists(stamp) and open(stamp).read() == version:
            return BIND
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    system = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
              cuda, sysconfig.get_paths()["include"]]
    tmp = BIND + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           f'-DWF_TORCH_VERSION="{version}"']
    for d in system:
        cmd += ["-isystem", d]
    cmd += [BIND_SRC, "-o", tmp, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {BIND_SRC} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(stamp, "w") as f:
        f.write(version)
    return BIND


def try_build_bind(force: bool = False, verbose: bool = False) -> str | None:
    """build_bind, or a report and no module: the library needs none, the row operators' calls only
    take more of the host's time. What an earlier build left may not fit the library any more."""
    try:
        return build_bind(force, verbose)
    except (RuntimeError, OSError, AttributeError) as e:
        if os.path.exists(BIND):
            os.remove(BIND)
        print(f"warning: the row operators' compiled binding was not built: {e}", file=sys.stderr, flush=True)
        return None


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            if f.endswith(".o"):
                os.remove(os.path.join(BUILD, f))
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, extra), srcs))
    if (not os.path.exists(LIB) or force or extra
            or max(os.path.getmtime(o) for o in objs) > os.path.getmtime(LIB)):
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + [
            "-lpthread", "-ldl", "-lrt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    try_build_bind(force, verbose)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra=extra))


if __name__ == "__main__":
    sys.exit(main())
