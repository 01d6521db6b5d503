"""Build the CUDA library ``libar_gb300.so`` in-tree, for sm_103a only.

Each ``csrc/*.cu`` file is compiled by its own nvcc process (in parallel),
then the objects are linked into one shared library next to this file.  The
extension module ``_native`` (``csrc/ar_python.c``) is built beside it against
that library for the running interpreter, whose tag is in its file name; without
Python's headers it is left out.  A rebuild happens only when a source or header
is newer than what was built.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libar_gb300.so")
NATIVE = os.path.join(HERE, "_native" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
NATIVE_SOURCE = os.path.join(CSRC, "ar_python.c")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    # IEEE arithmetic: no flush to zero, no fast math (the fold must match
    # the binary32 round-to-nearest definition bit for bit)
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-I" + INCLUDE, "-I" + CSRC,
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newest(files: list[str]) -> float:
    return max(os.path.getmtime(f) for f in [*files, os.path.abspath(__file__)])


def _fresh(built: str, newest: float) -> bool:
    return os.path.exists(built) and os.path.getmtime(built) >= newest


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
    if res.stderr.strip():
        sys.stderr.write(res.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link what is needed; returns the library's path."""
    headers = glob.glob(os.path.join(INCLUDE, "*.h"))
    private = [f for end in ("*.h", "*.cuh") for f in glob.glob(os.path.join(CSRC, end))]
    if force or not _fresh(LIB, _newest(sources() + headers + private)):
        os.makedirs(BUILD, exist_ok=True)
        extra = ["-Xptxas", "-v"] if verbose_ptxas else []
        srcs = sources()
        with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
            objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        _link(LIB, [*objs, "-lcudart"])
    if force or not _fresh(NATIVE, _newest([NATIVE_SOURCE, *headers])):
        _build_native()
    return LIB


def _build_native() -> None:
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        sys.stderr.write("no Python.h in %s: the layer operators are called through ctypes, a few "
                         "us a call more\n" % include)
        return
    _link(NATIVE, ["-O2", "-Xcompiler", "-fPIC,-Wall,-Wextra", "-I" + INCLUDE, "-I" + include,
                   NATIVE_SOURCE, "-L" + HERE, "-lar_gb300", "-Xlinker", "-rpath=$ORIGIN",
                   "-cudart", "none"])


def _link(out: str, args: list[str]) -> None:
    tmp = out + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *args]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    if res.stderr.strip():
        sys.stderr.write(res.stderr)
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
