"""Build libkmip.so (CUDA, sm_100a) in-tree with nvcc.

    python -m graph_transformer_sparse_kmip_b200.build [--force] [--jobs N]

Each ``csrc/*.cu`` compiles to an object under ``_build/`` (skipped when the
object is newer than every source and header), then all objects link into
``graph_transformer_sparse_kmip_b200/libkmip.so`` with the CUDA runtime
linked statically, so the library needs only the driver at run time.
``csrc/kmip_host.cpp`` becomes ``_kmip_host-<tag>.so``, the module through which
binding.py calls the operators around the attention (g++, torch's headers).  It
holds inline code of torch and of CPython, so the tag names their versions
(host_path), and a module built for others is neither kept nor loaded.

``--debug-bounds`` builds ``libkmip_debug.so`` instead (objects under
``_build/debug/``) with KMIP_DEBUG_BOUNDS defined: the kernels then check
every key index they are about to read against the query's graph and record
KMIP_ERR_BAD_INDEX in the status word instead of reading out of range.  The
binding loads it when KMIP_DEBUG_BOUNDS=1.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import hashlib
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkmip.so")
LIB_DEBUG = os.path.join(PKG, "libkmip_debug.so")
NVCC = os.environ.get("NVCC", "nvcc")
CXX = os.environ.get("CXX", "g++")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++20", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _compile(src: str, force: bool, verbose: bool, debug: bool = False) -> str:
    obj = os.path.join(BUILD, "debug" if debug else "", os.path.basename(src)[:-3] + ".o")
    newest = max(os.path.getmtime(p) for p in [src] + _headers())
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    cmd = [NVCC, *ARCH, *FLAGS, *(["-DKMIP_DEBUG_BOUNDS"] if debug else []), "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def host_path() -> str:
    """The host module for this interpreter and this torch."""
    import torch
    made_for = (torch.__version__, torch.version.cuda, torch.version.git_version,
                torch.compiled_with_cxx11_abi(), sysconfig.get_config_var("SOABI"))
    tag = hashlib.sha1(repr(made_for).encode()).hexdigest()[:12]
    return os.path.join(PKG, f"_kmip_host-{tag}.so")


def _build_host(force: bool) -> None:
    src, host = os.path.join(CSRC, "kmip_host.cpp"), host_path()
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(ROOT, "include", "kmip.h")))
    if not force and os.path.exists(host) and os.path.getmtime(host) >= newest:
        return
    import torch
    from torch.utils import cpp_extension
    dirs = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"],
            *cpp_extension.include_paths(device_type="cuda")]
    tmp = f"{host}.{os.getpid()}.tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f for d in dirs for f in ("-isystem" if "torch" in d else "-I", d)), src, "-o", tmp,
           *(f"-L{d}" for d in cpp_extension.library_paths()), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, host)
    for old in glob.glob(os.path.join(PKG, "_kmip_host*.so")):
        if old != host:
            os.remove(old)


def build(force: bool = False, jobs: int | None = None, verbose: bool = False,
          debug_bounds: bool = False) -> str:
    os.makedirs(os.path.join(BUILD, "debug") if debug_bounds else BUILD, exist_ok=True)
    lib = LIB_DEBUG if debug_bounds else LIB
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, os.cpu_count() or 1)) as ex:
        host = ex.submit(_build_host, force)
        objs = list(ex.map(lambda s: _compile(s, force, verbose, debug_bounds), srcs))
        host.result()
    if force or not os.path.exists(lib) or os.path.getmtime(lib) < max(os.path.getmtime(o) for o in objs):
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", lib, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--jobs", type=int, default=None)
    ap.add_argument("-v", "--verbose", action="store_true", help="print ptxas resource usage")
    ap.add_argument("--debug-bounds", action="store_true",
                    help="build libkmip_debug.so with device-side index checks")
    args = ap.parse_args()
    print(build(force=args.force, jobs=args.jobs, verbose=args.verbose,
                debug_bounds=args.debug_bounds))
