"""Build libkvd.so in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel into ``_build/`` and is linked
into ``decode_attention_kv_gb300/libkvd.so`` (CUDA runtime linked
statically).  The host binding of the latent and the serving-step calls
(csrc/binding) compiles beside them against the installed torch, into a file named
for that torch and this Python.  libkvd.so needs nvcc only: where the binding does
not compile, the build goes on without it and those calls raise what stopped it.
Rebuilds only when a source or header is newer than the libraries.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvd.so")
BINDING_SRC = os.path.join(CSRC, "binding", "latent_binding.cpp")
BINDING_ERROR = os.path.join(BUILD, "latent_binding.error")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA toolkit required to build libkvd)")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) +
                  glob.glob(os.path.join(CSRC, "*", "*.cu")))


def _inputs():
    return sources() + [p for d in ("", "*") for e in ("*.cuh", "*.h")
                        for p in glob.glob(os.path.join(CSRC, d, e))] + [
        os.path.join(ROOT, "include", "kvd.h"), __file__]


def _newer(lib, inputs) -> bool:
    return os.path.exists(lib) and all(
        os.path.getmtime(p) <= os.path.getmtime(lib) for p in inputs)


def binding_path() -> str:
    """The binding's file for the installed torch and this Python: tensors are read
    through torch's own types, whose layout goes with its version and C++ ABI."""
    import torch
    return os.path.join(PKG, "_latent_binding.torch-{}.abi{}.{}.so".format(
        torch.__version__, int(torch._C._GLIBCXX_USE_CXX11_ABI), sysconfig.get_config_var("SOABI")))


def up_to_date() -> bool:
    """libkvd.so is as new as its sources."""
    return _newer(LIB, _inputs())


def binding_up_to_date() -> bool:
    """So is the binding, and it was compiled against the installed torch."""
    return _newer(binding_path(), [BINDING_SRC, os.path.join(ROOT, "include", "kvd.h"), __file__])


def build_binding() -> str:
    """Compile the host binding of the latent and serving-step calls; returns its path."""
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = binding_path()
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        cmd += ["-isystem", d]
    cmd += [BINDING_SRC, "-o", tmp, "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def _try_binding(force: bool) -> None:
    """The binding, if it compiles here; what stops it is kept for its calls."""
    try:
        if force or not binding_up_to_date():
            build_binding()
        error = None
    except Exception as e:  # no g++, no headers, no torch: libkvd.so is none the worse
        error = f"{type(e).__name__}: {e}"
        print(f"warning: the latent calls will not run, their binding does not compile: {error}",
              file=sys.stderr)
    if error is not None:
        os.makedirs(BUILD, exist_ok=True)
        with open(BINDING_ERROR, "w") as f:
            f.write(error)
    elif os.path.exists(BINDING_ERROR):
        os.remove(BINDING_ERROR)


def binding_error() -> str:
    """What stopped the last build of the binding, or how to build it."""
    if os.path.exists(BINDING_ERROR):
        with open(BINDING_ERROR) as f:
            return f.read()
    return "build it first (python -c 'import __graft_entry__ as g; g.build()')"


def build(force: bool = False, verbose: bool = False, jobs: int | None = None,
          extra_flags: list[str] | None = None) -> str:
    """Compile and link libkvd.so, and the binding if it compiles; returns libkvd.so's path."""
    if not force and up_to_date():
        _try_binding(False)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = FLAGS + (extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *flags, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_try_binding, force)
        objs = list(ex.map(compile_one, srcs))
        binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
