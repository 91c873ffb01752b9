"""Build libtlgemm.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc,
and its checked twin libtlgemm_checked.so (-DTL_CHECKED: the kernels test their
index invariants at run time and report a violation in the device error word;
used by the tests, never by the product path).

    python tensor_core_gemm_tl_b200/build.py [--force] [--verbose-ptxas] [--checked]

(Run as a script: importing the package loads the library it builds.)
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtlgemm.so")
CHECKED_LIB = os.path.join(PKG, "libtlgemm_checked.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.inc"))
                              + glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in inputs())


def _compile(src: str, obj: str, force: bool, flags) -> None:
    """One source to an object; kept when the same command made it and it is newer
    than everything that compile read (nvcc's own dependency list and the
    command lie beside the object)."""
    deps, made_by = obj + ".d", obj + ".cmd"
    command = [NVCC, *flags, "-I", INCLUDE, "-I", CSRC, "-c", src]
    if not force and all(os.path.exists(f) for f in (obj, deps, made_by)):
        with open(deps) as fh:
            read = fh.read().split(":", 1)[1].replace("\\\n", " ").split()
        with open(made_by) as fh:
            same = fh.read() == "\n".join(command)
        t = os.path.getmtime(obj)
        if same and all(os.path.exists(f) and os.path.getmtime(f) <= t for f in read):
            return
    tmp = obj + f".tmp{os.getpid()}"
    if os.path.exists(made_by):
        os.remove(made_by)  # until the object is the new command's
    subprocess.check_call([*command, "-MMD", "-MF", deps, "-o", tmp])
    os.replace(tmp, obj)
    with open(made_by, "w") as fh:
        fh.write("\n".join(command))


def build(force: bool = False, ptxas_verbose: bool = False, out: str = LIB, extra=()) -> str:
    if not force and not ptxas_verbose and not stale(out):
        return out
    objdir = os.path.join(ROOT, "build", os.path.basename(out))
    os.makedirs(objdir, exist_ok=True)
    flags = [f for f in NVCC_FLAGS if f != "-shared"] + list(extra) + (["-Xptxas", "-v"] if ptxas_verbose else [])
    objs = [os.path.join(objdir, os.path.basename(s) + ".o") for s in sources()]
    # the sources are independent: compile them side by side
    with ThreadPoolExecutor(max_workers=len(objs)) as pool:
        list(pool.map(lambda so: _compile(so[0], so[1], force, flags), zip(sources(), objs)))
    tmp = out + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *NVCC_FLAGS, "-o", tmp, *objs])
    os.replace(tmp, out)
    return out


def build_checked(force: bool = False) -> str:
    return build(force=force, out=CHECKED_LIB, extra=("-DTL_CHECKED",))


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--checked", action="store_true", help="also build libtlgemm_checked.so")
    a = ap.parse_args(argv)
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas))
    if a.checked:
        print(build_checked(force=a.force))


if __name__ == "__main__":
    sys.exit(main())
