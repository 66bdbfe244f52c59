"""Build the CUDA library in-tree: bit_blockwise_adamw_gb300/_build/libq8adamw.so.

Every translation unit is compiled by nvcc for sm_103a only, in parallel,
then linked into one shared library that exports the C ABI of
include/q8adamw.h.  Floating-point contraction is off (--fmad=false): each
fp32 operation of the step rounds on its own.  Beside it goes a small CPython
module of the binding (csrc/q8_lists.cpp, g++ and torch's headers), for the
installed torch; where that does not compile, the library is built all the same,
and the binding's calls on lists of gradients say that the module is missing.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libq8adamw.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--fmad=false",
                     "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "-I", INCLUDE, "-I", CSRC]


def lists_module():
    """Path of the CPython module of csrc/q8_lists.cpp, which holds for one version of torch and of Python."""
    import torch
    return os.path.join(OUT_DIR, "q8_lists-%s-%s" % (torch.__version__, sysconfig.get_config_var("EXT_SUFFIX").lstrip(".")))


def _build_lists(force):
    try:
        _compile_lists(force)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn("q8_lists is not built, and q8_grad_norm and q8_clip_grads cannot be called from Python: %s" % e, RuntimeWarning)


def _compile_lists(force):
    import torch
    src, out = os.path.join(CSRC, "q8_lists.cpp"), lists_module()
    inputs = [src, os.path.join(INCLUDE, "q8train.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(map(os.path.getmtime, inputs)):
        return
    root = os.path.dirname(os.path.abspath(torch.__file__))
    tmp = out + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-unknown-pragmas",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], src, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        os.replace(tmp, out)
    except (OSError, RuntimeError):
        if os.path.exists(out):
            os.remove(out)                               # of older sources
        raise


def nvcc():
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda_home, "bin", "nvcc")
    return path if os.path.exists(path) else (shutil.which("nvcc") or "nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library if any input changed; return its path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and not _stale():
        _build_lists(False)
        return LIB
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 4)) as ex:
        lists = ex.submit(_build_lists, force)
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    lists.result()
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else []))
