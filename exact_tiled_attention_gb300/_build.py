"""Builds libgbattn.so in-tree with nvcc for sm_103a (no CMake, no torch
extension machinery): each .cu compiles in parallel, then one link step.  The
compiled half of the Python binding (C++ against the installed PyTorch's headers)
is built beside it; its file is named after the Python and the PyTorch that it is
for, so one built for others is not loaded.

    python -m exact_tiled_attention_gb300._build [--force] [--verbose]
    python exact_tiled_attention_gb300/_build.py     # the C library, without PyTorch

Build option (environment): GBATTN_EX2_EMU_EVERY=E evaluates every E-th pair
of softmax exponentials with the FMA-pipe polynomial instead of the MUFU unit
(default 0 = none; the library is rebuilt when the setting changes).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgbattn.so")
EXT_SOURCE = "paged_binding.cpp"

SOURCES = ["gbattn_api.cu", "prefill_fwd.cu", "prefill_pair.cu", "prefill_fp8.cu", "decode_splitkv.cu",
           "decode_noalloc.cu", "backward.cu", "backward_atomic.cu",
           "gbattn_api_cache.cu", "qk_norm_rope.cu", "cache_pages.cu", "decode_paged.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _deps() -> list[str]:
    out = [os.path.join(INCLUDE, "gbattn.h")]
    for f in os.listdir(CSRC):
        if f != EXT_SOURCE:
            out.append(os.path.join(CSRC, f))
    return out


def _ext_deps() -> list[str]:
    return [os.path.join(INCLUDE, "gbattn.h"), os.path.join(CSRC, EXT_SOURCE)]


def ext_path() -> str:
    """Where the binding's compiled half for this Python and this PyTorch belongs."""
    import torch

    return os.path.join(PKG, f"_paged-{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}.so")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _options() -> list[str]:
    emu = int(os.environ.get("GBATTN_EX2_EMU_EVERY", "0") or 0)
    return [f"-DGBATTN_EX2_EMU_EVERY={emu}"]


def _ext_commands(path: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of the binding's compiled half at `path`."""
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, EXT_SOURCE.replace(".cpp", ".o"))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                "-I", INCLUDE, "-isystem", sysconfig.get_path("include"), "-isystem", os.path.join(base, "include"),
                "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
                "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
    link = [cxx, "-shared", obj, "-o", path, "-L" + PKG, "-l:libgbattn.so",
            "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]
    return compile_, link


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed")


def _build_ext(path: str, verbose: bool) -> None:
    """Links the compiled half, whose object is there, against the library."""
    tmp = path + f".tmp{os.getpid()}"
    _run(_ext_commands(tmp)[1], "g++ link", verbose)
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Builds what is not up to date: the library, which needs nvcc and its host
    compiler only, and beside it the binding's compiled half where PyTorch is
    installed.  A failure of the second leaves the first in place."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "options.txt")
    opts = _options()
    old = open(stamp).read() if os.path.exists(stamp) else ""
    lib_stale = force or _stale(LIB, _deps()) or old != " ".join(opts)
    try:
        ext = ext_path()
    except ImportError:
        ext = None
        sys.stderr.write("PyTorch is not installed: building the C library alone, without its Python binding\n")
    ext_stale = ext is not None and (force or _stale(ext, _ext_deps()))
    if not lib_stale and not ext_stale:
        return LIB
    cc = nvcc() if lib_stale else ""
    extra = (["-Xptxas", "-v"] if ptxas_verbose else []) + opts

    def compile_one(src: str):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    sources = SOURCES if lib_stale else []
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        ext_object = pool.submit(_run, _ext_commands(ext)[0], f"g++ on {EXT_SOURCE}", verbose) if ext_stale else None
        results = list(pool.map(compile_one, sources))
    if lib_stale:
        for src, _, r in results:
            if verbose or ptxas_verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}")
        tmp = LIB + f".tmp{os.getpid()}"
        link = [cc, *ARCH, "-shared", "-o", tmp, *[obj for _, obj, _ in results]]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
        with open(stamp, "w") as f:
            f.write(" ".join(opts))
    if ext_stale:
        ext_object.result()
        _build_ext(ext, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)
