"""Build the CUDA library in-tree: csrc/*.cu -> _lib/libattn_gb300.so (sm_103a),
and the torch binding of its short calls: csrc/binding.cpp -> _lib/_native.so.

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library with the CUDA runtime linked statically.  The binding is compiled
beside them by the host compiler against the installed torch's headers, where they are.
Rebuilds only what changed (object newer than its source and the shared headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libattn_gb300.so")
NATIVE = os.path.join(OUT_DIR, "_native.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the attention library needs the CUDA toolkit to build")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "attn.h")]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _env_flags():
    """Extra nvcc flags from ATTN_NVCC_FLAGS (tuning builds, e.g. -DATTN_FWD_STAGES_D128=4)."""
    return os.environ.get("ATTN_NVCC_FLAGS", "").split()


def _compile(src: str, extra) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *_env_flags(), *extra, "-c", src, "-o", obj + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        os.replace(obj + ".tmp", obj)
    return obj


def _torch_dir() -> str | None:
    """The installed torch package's folder, without importing it."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _binding(force: bool) -> bool:
    """Builds the torch binding.  False: torch's or Python's headers, or a host compiler, are not
    here; the library does without (the Python binding makes the same calls, slower)."""
    src = os.path.join(CSRC, "binding.cpp")
    torch, cxx = _torch_dir(), shutil.which(os.environ.get("CXX") or "g++")
    python = sysconfig.get_paths()["include"]
    needs = [os.path.join(torch or "", "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(torch or "", "include", "c10", "cuda", "CUDAStream.h"), os.path.join(python, "Python.h")]
    if torch is None or cxx is None or not all(os.path.exists(n) for n in needs):
        if os.path.exists(NATIVE):
            os.remove(NATIVE)  # it may be another torch's
        return False
    # built anew when another torch is installed
    deps = [src, os.path.join(ROOT, "include", "attn.h"), os.path.join(torch, "version.py")]
    if not force and not _stale(NATIVE, deps):
        return True
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           python, os.path.join(cuda, "include")]
    lib = os.path.join(torch, "lib")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *(x for i in inc for x in ("-I", i)), src, "-o", NATIVE + ".tmp", "-L", lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the torch binding failed to build:\n{r.stdout}\n{r.stderr}")
    os.replace(NATIVE + ".tmp", NATIVE)
    return True


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(OBJ_DIR, "*.o")):
            os.remove(o)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_binding, force)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        if not binding.result():
            print("the torch binding of short calls is not built (it needs torch's and Python's headers and a "
                  "host compiler); calls take the Python binding", file=sys.stderr)
    if force or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs, "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
        if verbose:
            print("built", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
