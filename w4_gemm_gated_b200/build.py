"""Build the CUDA library ``libspear.so`` in-tree for sm_100a, and the native
marshalling module ``_bind`` of its binding (host code, against torch's headers).

Usage: ``python -m w4_gemm_gated_b200.build [--force] [--verbose] [--checked]``.
Objects go to ``_build/`` at the repository root; the shared library is
written next to this file so that it travels with the source tree.
``--checked`` builds the device-check variant ``libspear_checked.so`` (the
same sources with -DSPEAR_DEVICE_CHECKS; objects in ``_build/checked``).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libspear.so")
LIB_CHECKED = os.path.join(PKG, "libspear_checked.so")
BIND = os.path.join(PKG, "_bind" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
SOURCES = ["api.cu", "pack.cu", "decode.cu", "decode2.cu", "decode3.cu", "ec.cu", "tc_gemm.cu", "noalloc.cu",
           "kv_cache.cu", "attn_decode.cu", "block_norm.cu"]
HEADERS = ["common.cuh", "kernels.h", "tma.cuh", "kv_cache.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "spear.h")]
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str, verbose: bool, checked: bool = False) -> tuple[str, str]:
    odir = os.path.join(BUILD, "checked") if checked else BUILD
    obj = os.path.join(odir, os.path.splitext(src)[0] + ".o")
    extra = ["-DSPEAR_DEVICE_CHECKS"] if checked else []
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o",
           obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    log = res.stderr if verbose else ""
    return obj, log


def torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package
        import torch
        return str(torch.__version__)


def build_bind(force: bool = False) -> str:
    """The binding's native module; its CUDA side is reached through addresses
    handed to it, so it links to torch alone: to the C++ of one version, which
    a file in the objects' folder names."""
    src, header = os.path.join(CSRC, "bind.cpp"), os.path.join(ROOT, "include", "spear.h")
    mark, version = os.path.join(BUILD, "bind.torch"), torch_version()
    if not force and os.path.exists(BIND) and os.path.exists(mark):
        with open(mark) as f:
            built_for = f.read()
        if built_for == version and os.path.getmtime(BIND) >= max(os.path.getmtime(src), os.path.getmtime(header)):
            return BIND
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
                os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
                sysconfig.get_paths()["include"]]
    tmp = f"{BIND}.{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in includes], src,
           "-o", tmp, "-L" + os.path.join(base, "lib"),
           *["-l" + l for l in ("c10", "c10_cuda", "torch_cpu", "torch_cuda", "torch_python", "torch")]]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for bind.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BIND)
    os.makedirs(BUILD, exist_ok=True)
    with open(mark, "w") as f:
        f.write(version)
    return BIND


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    build_bind(force)
    lib = LIB_CHECKED if checked else LIB
    os.makedirs(os.path.join(BUILD, "checked") if checked else BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if not force and os.path.exists(lib):
        newest = max([os.path.getmtime(s) for s in srcs] + [_deps_mtime(), os.path.getmtime(__file__)])
        if os.path.getmtime(lib) >= newest:
            return lib
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose, checked), SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = lib + ".tmp"
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC", *objs,
           "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib)
    return lib


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--checked", action="store_true", help="build the device-check variant")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose, checked=args.checked))


if __name__ == "__main__":
    main()
