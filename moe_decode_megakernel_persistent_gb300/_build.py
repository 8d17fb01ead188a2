"""In-tree build of libmk.so (the C-ABI library) with nvcc for sm_103a, and of
the Python module _torch (tensor calls on it) with the host compiler.

The translation units compile in parallel (the decode kernel's file once
per group of its instantiations, MK_KERNEL_PART 0..3); the shared objects
land next to this file.  Rebuilds only what is older than its sources, the
module also when another torch or Python is installed than it was built for.
libmk.so needs nvcc alone: it is in place whatever becomes of the module,
which is left out where there is no torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmk.so")
MODULE = os.path.join(PKG, "_torch.so")
BUILD = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
              "-I" + CSRC]
# (source, object name, extra flags)
SOURCES = [("mk_kernel.cu", f"mk_kernel_p{p}", [f"-DMK_KERNEL_PART={p}"]) for p in range(4)] + [
    (f, os.path.splitext(f)[0], []) for f in ("mk_host.cpp", "mk_static.cu", "mk_pack.cu", "mk_kv.cu", "mk_kv4.cu", "mk_kv4_attention.cu",
                                                  "mk_kv4_wide.cu", "mk_pages.cu", "mk_paged.cu", "mk_paged_attention.cu",
                                                  "mk_paged_wide.cu", "mk_paged_mass.cu", "mk_paged_evict.cu", "mk_prefill.cu")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


MODULE_SOURCE = "mk_torch.cpp"


def _inputs(module: bool):
    files = [MODULE_SOURCE] if module else [f for f in os.listdir(CSRC) if f != MODULE_SOURCE]
    return [os.path.join(CSRC, f) for f in files] + [os.path.join(INCLUDE, "mk.h"), os.path.abspath(__file__)]


def _built_for():
    """What the module is compiled against: this Python and the installed torch; None without one."""
    try:
        return f"{sys.implementation.cache_tag} torch {importlib.metadata.version('torch')}"
    except importlib.metadata.PackageNotFoundError:
        return None


def _stamp() -> str:
    return os.path.join(BUILD, "mk_torch.for")


def _newer(path: str, files) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def _lib_current() -> bool:
    return _newer(LIB, _inputs(False))


def _module_current() -> bool:
    built_for = _built_for()
    if built_for is None:
        return True  # there is none to build
    if not _newer(MODULE, _inputs(True)) or not os.path.exists(_stamp()):
        return False
    with open(_stamp()) as f:
        return f.read() == built_for


def up_to_date() -> bool:
    return _lib_current() and _module_current()


def _module_commands(obj: str, out: str) -> list:
    """The host compiler's two commands for the Python module: against the
    installed torch, this interpreter and libmk.so next to it."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    cxx, cuda = os.environ.get("CXX", "g++"), os.path.dirname(os.path.dirname(_nvcc()))
    inc = [f"-I{d}" for d in (*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE)]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return [[cxx, "-O2", "-std=c++17", "-fPIC", abi, *inc, "-c", os.path.join(CSRC, "mk_torch.cpp"), "-o", obj],
            [cxx, "-shared", obj, "-o", out, "-L" + os.path.dirname(LIB), "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L" + libs,
             "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda"]]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libmk.so if needed; returns its path.  Raises on failure."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(item):
        src, name, extra = item
        obj = os.path.join(BUILD, name + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra]
        if src.endswith(".cu") and verbose:
            cmd += ["-Xptxas", "-v"]
        cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-6000:]}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stderr[-6000:]}")

    def build_lib():
        with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
            objs = list(ex.map(compile_one, SOURCES))
        # cuBLAS (the chunked prefill's GEMMs) is found through the toolkit's
        # library directory
        cudalib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", LIB + ".tmp", *objs, "-lcublas",
             "-Xlinker", "-rpath=" + cudalib], "link")
        os.replace(LIB + ".tmp", LIB)

    def compile_module():
        commands = _module_commands(os.path.join(BUILD, "mk_torch.o"), MODULE + ".tmp")
        run(commands[0], "the Python module's compilation")
        return commands[1]

    with cf.ThreadPoolExecutor(1) as ex:
        module = ex.submit(compile_module) if _built_for() and (force or not _module_current()) else None
        if force or not _lib_current():
            build_lib()
        if module:
            run(module.result(), "the Python module's link")
            os.replace(MODULE + ".tmp", MODULE)
            with open(_stamp(), "w") as f:
                f.write(_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
