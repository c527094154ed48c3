"""Build libsscan.so (the CUDA library behind include/sscan.h) in-tree for sm_100a."""
import concurrent.futures
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsscan.so")
# the same library with the index checks of csrc/sscan_check.cuh compiled in
LIB_DEBUG = os.path.join(HERE, "libsscan_debug.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                              + glob.glob(os.path.join(ROOT, "include", "*.h")))


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile every .cu under csrc/ into one shared library (sm_100a only).

    debug=True builds libsscan_debug.so instead: the same kernels with every computed
    index into a workspace, parameter or state array checked (SSCAN_DEBUG_BOUNDS); a bad
    index raises bit 3 of the device status word and the access is skipped.  It is
    compiled with relocatable device code so that all kernels share that word."""
    out = LIB_DEBUG if debug else LIB
    if not force and os.path.exists(out):
        newest = max(os.path.getmtime(p) for p in deps())
        if os.path.getmtime(out) >= newest:
            return out
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if debug:
        flags += ["-DSSCAN_DEBUG_BOUNDS=1", "-rdc=true"]
    if verbose:
        flags.append("-Xptxas=-v")
    # one object per source, compiled side by side; an object newer than its source and
    # every header is kept
    objdir = os.path.join(HERE, "_build", "debug" if debug else "release")
    os.makedirs(objdir, exist_ok=True)
    headers = max(os.path.getmtime(p) for p in deps() if not p.endswith(".cu"))

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        if force or not os.path.exists(obj) or os.path.getmtime(obj) <= max(headers, os.path.getmtime(src)):
            subprocess.run([NVCC, *flags, "-c", src, "-o", obj + ".tmp"], check=True)
            os.replace(obj + ".tmp", obj)
        return obj

    with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objects = list(pool.map(compile_one, sources()))
    subprocess.run([NVCC, *flags[:2], "-shared", *(["-rdc=true"] if debug else []), "-o", out + ".tmp", *objects], check=True)
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
