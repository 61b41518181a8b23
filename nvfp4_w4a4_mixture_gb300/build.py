"""Build libmoe_nvfp4.so (in-tree, under nvfp4_w4a4_mixture_gb300/_lib/) for sm_103a with nvcc.

One nvcc process per translation unit, run in parallel, then one link step. The library links
the CUDA runtime statically and looks up the driver's tensor-map encoder at run time, so it needs
no libcuda at link time.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
SRC_DIR = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(OUT_DIR, "obj")
LIB = os.path.join(OUT_DIR, "libmoe_nvfp4.so")
CALLS_SRC = os.path.join(SRC_DIR, "calls.c")
CALLS = os.path.join(OUT_DIR, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I" + INCLUDE]


def _nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(glob.glob(os.path.join(SRC_DIR, "*.cu")))


def _deps_mtime():
    files = sources() + glob.glob(os.path.join(SRC_DIR, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(f) for f in files)


def build_calls(force: bool = False) -> None:
    """The C marshalling of the block calls (calls.c), where Python's headers are installed; without it the
    same calls go through ctypes."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return
    newest = max(os.path.getmtime(f) for f in [CALLS_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))
    if not force and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= newest:
        return
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = CALLS + ".tmp.%d" % os.getpid()
    cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + include, "-I" + INCLUDE, CALLS_SRC, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("gcc failed for %s:\n%s\n%s" % (CALLS_SRC, r.stdout, r.stderr))
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False) -> str:
    build_calls(force)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc] + ARCH + FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose:
        for obj, log in results:
            print(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
