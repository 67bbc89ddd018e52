"""Build ``libpa.so`` (the C-ABI paged-attention library) for sm_103a.

Each ``csrc/*.cu`` file is compiled in parallel with nvcc, then linked into a
shared library with the CUDA runtime linked statically, so the library only
needs the driver at run time.  Output: ``paged_kv_cache_193_gb300/_build/libpa.so``.
Beside it ``csrc/binding.cpp`` becomes ``_pa_binding.so``, the CPython binding
of the calls whose kernels are shorter than a check of their arguments in
Python.  The library needs no torch; without one that has CUDA the binding
alone is left out.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpa.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(OUT_DIR, "_pa_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _sources() + _headers() + [__file__])


def compile_flags(verbose_ptxas: bool = False) -> list[str]:
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I" + INCLUDE, "-I" + CSRC, "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    return flags


def binding_for(torch) -> str:
    """What a binding built now fits: it uses C++ interfaces of torch, which
    change between versions, and Python's.  Kept beside it in a ``.for`` file."""
    return f"torch {torch.__version__}, Python {sysconfig.get_config_var('SOABI')}"


def built_for(binding: str) -> str:
    try:
        with open(binding + ".for") as f:
            return f.read()
    except FileNotFoundError:
        return "unknown"


def build_binding(force: bool = False) -> str:
    """Compile the CPython binding if its source is newer, or it was built for
    another torch; return its path.  Raises ImportError without a torch that
    has CUDA."""
    import torch
    newest = max(os.path.getmtime(f) for f in [BINDING_SRC, *_headers(), __file__])
    if (not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest
            and built_for(BINDING) == binding_for(torch)):
        return BINDING
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    if not os.path.exists(os.path.join(lib, "libc10_cuda.so")):
        raise ImportError(f"the torch in {root} has no CUDA")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the binding failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if os.path.exists(BINDING + ".for"):
        os.remove(BINDING + ".for")  # says nothing while the two do not belong together
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(binding_for(torch))
    os.replace(tmp, BINDING + ".for")
    return BINDING


def _finish(binding) -> None:
    """The result of ``build_binding``: what it needs of torch may be missing,
    anything else that fails is raised."""
    try:
        binding()
    except ImportError as e:
        sys.stderr.write(f"{BINDING} not built ({e}): the calls of the library itself are all there, "
                         "the Python calls that go through the binding are not\n")


def build(force: bool = False, verbose_ptxas: bool = False, out: str | None = None,
          defines: tuple[str, ...] = ()) -> str:
    """Compile and link if any source is newer than the library; return its
    path.  ``out`` and ``defines`` (e.g. ``("PA_DECODE_WARPS=2",)``) build a
    variant of the library elsewhere, for launch-shape tuning."""
    lib = out or LIB
    if not force and not defines and out is None and not _stale():
        _finish(build_binding)
        return LIB
    obj_dir = os.path.join(os.path.dirname(lib), os.path.basename(lib) + ".objs") if out else OUT_DIR
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    flags = compile_flags(verbose_ptxas) + ["-D" + d for d in defines]

    def one(src: str) -> tuple[str, str]:
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(build_binding, force) if out is None else None
        results = list(ex.map(one, srcs))
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if binding is not None:
        _finish(binding.result)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
