"""In-tree build of the CUDA library (sm_103a), no CMake.

Compiles every ``csrc/*.cu`` to an object in parallel with nvcc, then links
``_build/liblagb300.so``. The library is a plain C ABI (``include/la.h``):
CUDA runtime linked statically, driver entry points resolved at run time,
so the shared object loads on a machine without a GPU: nvcc is all it takes.
``csrc/la_marshal.cpp``, which marshals the binding's most frequent calls, is compiled beside
them with g++ against the installed torch into ``_build/la_marshal.so`` (it reaches the library
through pointers), again for another torch or Python. Where torch is not installed it is left
out; where it does not compile the library is there all the same, and the build says so.
"""

import concurrent.futures as cf
import glob
import importlib.metadata
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


def _newer(built, *patterns):
    """Whether `built` exists and no file of the patterns is newer."""
    if not os.path.exists(built):
        return False
    files = [f for p in patterns for f in glob.glob(p)]
    return all(os.path.getmtime(f) <= os.path.getmtime(built) for f in (*files, os.path.abspath(__file__)))


def _lib_up_to_date():
    return _newer(LIB, *(os.path.join(CSRC, p) for p in ("*.cu", "*.cuh", "*.h")), os.path.join(ROOT, "include", "*.h"))


def _made_for():
    """The torch and the Python that la_marshal.so is made for (None: no torch)."""
    try:
        return f"torch {importlib.metadata.version('torch')}, {sys.implementation.cache_tag}"
    except importlib.metadata.PackageNotFoundError:
        return None


def _marshal_up_to_date():
    want = _made_for()
    if want is None:
        return True
    try:
        with open(MARSHAL + ".for") as f:
            made = f.read()
    except OSError:
        return False
    return made == want and _newer(MARSHAL, os.path.join(CSRC, "la_marshal.cpp"), os.path.join(ROOT, "include", "*.h"))


def up_to_date():
    return _lib_up_to_date() and _marshal_up_to_date()


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


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    return r.returncode, r.stdout + r.stderr


def _build_marshal():
    """Compiles la_marshal.so; the compiler's complaint if it does not."""
    out, made = MARSHAL + ".tmp", _made_for()
    try:
        rc, text = _run(_marshal_command(out))
    except (ImportError, AttributeError, OSError) as e:  # (a torch that does not load, no g++)
        return f"{type(e).__name__}: {e}"
    if rc != 0:
        return text
    os.replace(out, MARSHAL)
    with open(MARSHAL + ".for", "w") as f:
        f.write(made)
    return None


def _build_lib(ex, verbose, extra_flags):
    nvcc = _nvcc()
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    results = list(ex.map(lambda pair: _run([nvcc, *NVCC_FLAGS, *extra_flags, "-c", pair[0], "-o", pair[1]]),
                          zip(srcs, objs)))
    said = [f"--- {os.path.basename(s)}\n{out}" for s, (rc, out) in zip(srcs, results) if out.strip()]
    if verbose:
        sys.stderr.write("".join(said))
    failed = [f"--- {os.path.basename(s)}\n{out}" for s, (rc, out) in zip(srcs, results) if rc != 0]
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(failed))
    tmp = LIB + ".tmp"
    rc, out = _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"])
    if rc != 0:
        raise RuntimeError("link failed:\n" + out)
    os.replace(tmp, LIB)


def build(force=False, verbose=False, extra_flags=()):
    """Build what is older than its sources; returns the library's path."""
    lib, marshal = force or not _lib_up_to_date(), force and _made_for() is not None or not _marshal_up_to_date()
    if not lib and not marshal:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        pending = ex.submit(_build_marshal) if marshal else None
        if lib:
            _build_lib(ex, verbose, extra_flags)
        failed = pending.result() if pending else None
    if failed:
        raise RuntimeError(f"the library is built, {LIB}, but la_marshal.cpp, a part of the Python binding, is not:\n{failed}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
