"""In-tree build of the CUDA library (sm_103a), no CMake.

Compiles every ``csrc/*.cu`` to an object in parallel with nvcc, then links
``_build/liblagb300.so``. The library is a plain C ABI (``include/la.h``):
CUDA runtime linked statically, driver entry points resolved at run time,
so the shared object loads on a machine without a GPU. ``csrc/la_marshal.cpp``, which
marshals the binding's most frequent calls, is compiled beside them with g++ against the
installed torch into ``_build/la_marshal.so`` (it reaches the library through pointers).
"""

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "liblagb300.so")
MARSHAL = os.path.join(BUILD, "la_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "-I" + os.path.join(ROOT, "include"),
]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    pats = ("*.cu", "*.cuh", "*.h", "*.cpp")
    files = [f for p in pats for f in glob.glob(os.path.join(CSRC, p))]
    files += glob.glob(os.path.join(ROOT, "include", "*.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date():
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return all(os.path.getmtime(f) <= t for f in _deps())


def _marshal_command(out):
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           sysconfig.get_paths()["include"]]
    libs = os.path.join(home, "lib")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f for p in inc for f in ("-isystem", p)], "-I" + os.path.join(ROOT, "include"),
            os.path.join(CSRC, "la_marshal.cpp"), "-o", out, "-L" + libs, "-Wl,-rpath," + libs,
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]


def build(force=False, verbose=False, extra_flags=()):
    """Build the shared library if any source is newer; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = (_marshal_command(obj) if src.endswith(".cpp")
               else [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj])
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r.returncode, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        pairs = [(os.path.join(CSRC, "la_marshal.cpp"), MARSHAL + ".tmp"), *zip(srcs, objs)]
        results = list(ex.map(compile_one, pairs))
    failed = [(s, out) for s, rc, out in results if rc != 0]
    for s, rc, out in results:
        if verbose and out.strip():
            sys.stderr.write(f"--- {os.path.basename(s)}\n{out}")
    if failed:
        msg = "\n".join(f"--- {os.path.basename(s)}\n{out}" for s, out in failed)
        raise RuntimeError("compilation failed:\n" + msg)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    os.replace(MARSHAL + ".tmp", MARSHAL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
