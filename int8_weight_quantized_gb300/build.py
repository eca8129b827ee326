"""Build the CUDA library libck_int8.so in-tree, for sm_103a only, and the compiled part of
its Python binding.

Each .cu file is compiled by its own nvcc process (in parallel), then the objects are
linked into one shared library with the CUDA runtime linked statically, so the
library has no dependency beyond the driver.  The result lives next to this file
(``lib/libck_int8.so``); the Python binding loads it from there.  ``lib/_ck_binding.so``
(csrc/binding.cpp, compiled against the installed torch by the host compiler) hands tensors
to the operators around the linear layers; where it does not compile, the library is built all
the same, and those operators say that it is missing.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libck_int8.so")
BINDING = os.path.join(LIB_DIR, "_ck_binding.so")

SOURCES = ["api.cu", "quantize.cu", "gemm.cu", "api_transformer.cu", "norm_rope.cu", "paged_attention.cu",
           "attention.cu", "int4.cu"]
HEADERS = ["ck_device.cuh", "ck_internal.h", "gemm_common.cuh", "api_common.h", "transformer.h", "attn_common.cuh",
           "warp_mma.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libck_int8.so")
    return cand


def _fresh(target, sources):
    """Whether target exists and is no older than its sources (of CSRC), the header and this file."""
    files = [os.path.join(CSRC, s) for s in sources] + [os.path.join(INCLUDE, "ck_int8.h"), __file__]
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(f) for f in files)


def _compile(src, verbose):
    obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj, r.stderr


def _compile_binding():
    """binding.cpp -> lib/_ck_binding.so, against the torch that will load it."""
    import sysconfig

    import torch
    top = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           "-isystem", os.path.join(top, "include"), "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-isystem", cuda, "-isystem", "/usr/local/cuda/include", "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(top, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(top, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for binding.cpp:\n%s\n%s" % (cmd[0], r.stdout, r.stderr))
    os.replace(tmp, BINDING)


def _compile_library(verbose):
    with cf.ThreadPoolExecutor(max_workers=max(1, len(SOURCES))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)


def build(force=False, verbose=False, require_binding=False):
    """Compile what is older than its sources; return the library path.  A binding that does not
    compile is reported on stderr and left out, or with require_binding raised, after the library."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    failure = None
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = None if not force and _fresh(BINDING, ["binding.cpp"]) else ex.submit(_compile_binding)
        if force or not _fresh(LIB, SOURCES + HEADERS):
            _compile_library(verbose)
        if binding is not None:
            failure = binding.exception()
    if failure is not None:
        if os.path.exists(BINDING):  # of other sources
            os.remove(BINDING)
        if require_binding:
            raise failure
        sys.stderr.write("the operators around the linear layers are left out: %s\n" % failure)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
