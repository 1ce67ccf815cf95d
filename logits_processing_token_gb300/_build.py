"""In-tree build of libtg.so with nvcc for sm_103a (no cmake, no torch extension).

The library is plain CUDA C++ behind the C ABI of include/tg.h; it links the
CUDA runtime statically, so it uses the same primary context as PyTorch.  It
needs nvcc alone.  The marshalling module of the Python binding is compiled
beside it where PyTorch and its headers are there; without it the binding's
Python checks pass the attention calls on.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libtg.so")
BINDING = os.path.join(BUILD, "tg_binding.so")  # native argument marshalling of the attention calls
BINDING_SOURCE = "tg_binding.cpp"
SOURCES = ["tg_kernels.cu", "tg_api.cu", "tg_beam.cu", "tg_attn_api.cu", "tg_append.cu", "tg_read.cu", "tg_finish.cu", "tg_step.cu",
           "tg_step_e4m3.cu", "tg_step_i8.cu", "tg_wide.cu", "tg_wide_e4m3.cu", "tg_wide_i8.cu", "tg_prompt.cu"]
HEADERS = ["tg_device.cuh", "tg_select_core.cuh", "tg_attn.cuh", "tg_tokens.cuh", "tg_step.cuh", "tg_wide.cuh", "tg_mma5.cuh", os.path.join("..", "..", "include", "tg.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtg")


def _older(target: str, deps) -> bool:
    """target is not there, or older than one of deps (names in CSRC)."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in (os.path.join(CSRC, d) for d in deps) if os.path.exists(d))


def _stale_library() -> bool:
    return _older(LIB, SOURCES + HEADERS)


def _binding_for() -> str | None:
    """What a marshalling module has to be compiled for here; None without PyTorch."""
    import sysconfig
    try:
        import torch
    except ImportError:
        return None
    return "%s, torch %s" % (sysconfig.get_config_var("SOABI"), torch.__version__)


def binding_current() -> bool:
    """The marshalling module is there, and was compiled for this Python and PyTorch."""
    try:
        with open(BINDING + ".for") as f:
            return os.path.exists(BINDING) and f.read() == _binding_for()
    except OSError:
        return False


def build_binding() -> str:
    """Compile the marshalling module against the installed PyTorch's headers (host code only)."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(base, "include"), os.path.join(base, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-fPIC", "-shared", "-std=c++17",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    cmd += ["-I" + d for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
                               sysconfig.get_paths()["include"])]
    cmd += [os.path.join(CSRC, BINDING_SOURCE), "-o", BINDING + ".tmp", "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the compiler failed for %s:\n%s\n%s" % (BINDING_SOURCE, " ".join(cmd), r.stderr))
    os.replace(BINDING + ".tmp", BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(_binding_for())
    return BINDING


def _try_binding() -> None:
    """build_binding() where it can be; a failure is reported and leaves the library's build alone."""
    if _binding_for() is None:
        return
    try:
        build_binding()
    except Exception as e:  # no compiler, no headers, a file that is not there
        sys.stderr.write("tg_binding.so was not built; the attention calls take the binding's slower Python checks: %s\n" % e)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile libtg.so, and the marshalling module, if a source changed; return the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    binding = force or _older(BINDING, [BINDING_SOURCE, HEADERS[-1]]) or not binding_current()
    if not force and not _stale_library():
        if binding:
            _try_binding()
        return LIB
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + NVCC_FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        return obj, r.stderr

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        if binding:
            ex.submit(_try_binding)
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
