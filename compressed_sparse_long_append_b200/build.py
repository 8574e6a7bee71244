"""Build libcsla.so (sm_100a) in-tree with nvcc.

    python compressed_sparse_long_append_b200/build.py [--force] [--ptxas-v]
    python compressed_sparse_long_append_b200/build.py --timeline OUT.so

The second form builds a separate library with the device timeline hooks
compiled in (-DCSLA_TIMELINE, csla_timeline_read/clear exported).

The library has no torch dependency: it is plain CUDA C++ behind the C ABI
of include/csla.h.  Kernels are compiled for sm_100a only.

The sources share device symbols (-rdc=true), but for those in ALONE: a
kernel that moves registers between its warps (setmaxnreg) has to be
compiled as a whole program, the compiler ignores the instruction otherwise.
Such a unit keeps a device error word of its own, which csla_device_error
reads too.  (The timeline build compiles them like the others, so it times
them without that split.)
"""
import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcsla.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "--expt-relaxed-constexpr",
    "-I" + os.path.join(ROOT, "include"),
]
ALONE = {"kv_attend.cu"}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + [os.path.join(ROOT, "include", "csla.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)


def _link(out, extra=(), shared=(), verbose=False):
    """Compile every source (in parallel) and link them into `out`; those in ALONE and not in `shared` as whole programs."""
    with tempfile.TemporaryDirectory(dir=PKG, prefix="_build") as d:
        def one(src):
            name = os.path.basename(src)
            obj = os.path.join(d, name + ".o")
            alone = name in ALONE and name not in shared
            mode = ["-DCSLA_UNIT_ALONE"] if alone else ["-rdc=true"]
            _run([NVCC, *FLAGS, *extra, *mode, "-c", "-o", obj, src], verbose)
            return obj
        with ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as pool:
            objs = list(pool.map(one, sources()))
        tmp = out + ".tmp%d" % os.getpid()
        _run([NVCC, *FLAGS, "-rdc=true", "-shared", "-o", tmp, *objs], verbose)
        os.replace(tmp, out)
    return out


def build(force=False, verbose=False, extra=()):
    if not force and not _stale():
        return LIB
    return _link(LIB, extra, verbose=verbose)


def build_timeline(out):
    return _link(out, ["-DCSLA_TIMELINE"], shared=ALONE)


if __name__ == "__main__":
    if "--timeline" in sys.argv:
        print(build_timeline(os.path.abspath(sys.argv[sys.argv.index("--timeline") + 1])))
        sys.exit(0)
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(extra), verbose=True, extra=extra))
