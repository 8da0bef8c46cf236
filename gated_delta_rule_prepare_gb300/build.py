"""Builds libkda.so in-tree from csrc/*.cu for sm_103a (nvcc, no cmake).

Each translation unit compiles in parallel; the shared library links against
the shared CUDA runtime so it shares one runtime with the host process.  The
binding's short calls (csrc/fast_calls.c) become a Python extension beside it (the host's C
compiler, no library; named after the interpreter it is for).  Where that cannot be
built, for lack of Python's headers for one, the calls take their forms in Python.
"""

from __future__ import annotations

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
LIB = os.path.join(OUT_DIR, "libkda.so")
FAST = os.path.join(OUT_DIR, "fast_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "lib64")


def _newer(path, *patterns) -> bool:
    """Whether `path` is there and no older than the files that match."""
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for x in patterns for p in glob.glob(x))


def _headers() -> str:
    return os.path.join(INCLUDE, "*.h")


def _library_up_to_date() -> bool:
    return _newer(LIB, os.path.join(CSRC, "*.cu"), os.path.join(CSRC, "*.h"), _headers())


def _fast_up_to_date() -> bool:
    return _newer(FAST, os.path.join(CSRC, "fast_calls.c"), _headers())


def up_to_date() -> bool:
    return _library_up_to_date() and _fast_up_to_date()


def build_fast() -> bool:
    """Builds the Python extension; False, with a warning, where that fails."""
    tmp = FAST + ".tmp%d" % os.getpid()
    try:
        r = subprocess.run([shutil.which("cc") or "gcc", "-O2", "-fPIC", "-shared",
                            "-I" + INCLUDE, "-I" + sysconfig.get_paths()["include"],
                            os.path.join(CSRC, "fast_calls.c"), "-o", tmp],
                           capture_output=True, text=True)
        problem = r.stdout + r.stderr if r.returncode else None
    except OSError as e:
        problem = str(e)
    if problem is None:
        os.replace(tmp, FAST)
        return True
    if os.path.exists(FAST):            # (an older one may not fit the library)
        os.remove(FAST)
    warnings.warn("fast_calls.c cannot be built; its calls take longer in Python:\n" + problem)
    return False


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    if force or not _fast_up_to_date():
        build_fast()
    if not force and _library_up_to_date():
        return LIB
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I" + INCLUDE, "-I" + CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    flags += list(extra_flags or [])
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        r = subprocess.run([nvcc] + flags + ["-c", src, "-o", obj], capture_output=True,
                           text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, err in results:
            print(err)
    tmp = LIB + ".tmp%d" % os.getpid()
    link = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results]
    link += ["-Xlinker", "-rpath," + _cuda_lib_dir()]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
