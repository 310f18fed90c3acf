"""Build libspecverify.so (nvcc, sm_103a) and the Python binding of the paged
cache (the host compiler; torch's and Python's headers) in-tree.  The library
is built and loaded without the binding, which only cache.py uses."""
import os
import re
import subprocess
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libspecverify.so")
SOURCES = [os.path.join(CSRC, f) for f in ("spec_verify.cu", "spec_cache.cu", "tree_attn.cu", "cache4.cu",
                                              "tree_attn4.cu", "page_select.cu")]
BINDING = os.path.join(CSRC, "binding.cpp")
HEADERS = [os.path.join(INCLUDE, f) for f in ("spec_verify.h", "spec_cache.h")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + HEADERS

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "--threads", "0"]


CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def nvcc():
    cand = os.path.join(CUDA, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _older(path, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def stale() -> bool:
    return _older(LIB, DEPS)


def native_path() -> str:
    """The binding for this Python and this torch: it reads their objects, whose
    layouts change from version to version."""
    tag = "%s.torch%s.abi%d" % (sysconfig.get_config_var("SOABI"), torch.__version__,
                                int(torch._C._GLIBCXX_USE_CXX11_ABI))
    return os.path.join(OUT_DIR, "_native.%s.so" % re.sub(r"[^\w.-]", "_", tag))


def binding_stale() -> bool:
    return _older(native_path(), [BINDING] + HEADERS)


def _run(cmd, out, verbose):
    tmp = out + ".tmp%d" % os.getpid()
    cmd = cmd + ["-o", tmp]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, out)


def _binding_cmd():
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(CUDA, "include"), INCLUDE]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + p for p in inc] + [BINDING]
            + ["-L" + os.path.join(base, "lib"), "-L" + OUT_DIR, "-l:libspecverify.so", "-lc10", "-lc10_cuda", "-ltorch_cpu",
               "-ltorch_python", "-Wl,-rpath,$ORIGIN"])


def build_library(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    if force or stale():
        _run([nvcc(), *NVCC_FLAGS, "-I" + INCLUDE, "-I" + CSRC, *SOURCES], LIB, verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Links against the library, which has to be there."""
    path = native_path()
    if force or binding_stale():
        _run(_binding_cmd(), path, verbose)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
