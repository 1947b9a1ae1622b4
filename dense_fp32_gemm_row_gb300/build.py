"""Compile libgemmf32.so in-tree for sm_103a with nvcc (no cmake, no torch).

    python -m dense_fp32_gemm_row_gb300.build            # build if stale
    python -m dense_fp32_gemm_row_gb300.build --force    # rebuild everything

Each ``csrc/*.cu`` translation unit is compiled in parallel into
``_build/<name>.o`` (ptxas register/spill report in ``_build/<name>.ptxas.txt``)
and the objects are linked, with the static CUDA runtime, into
``dense_fp32_gemm_row_gb300/libgemmf32.so``.  ``csrc/binding/tensors.cpp``, the
Python binding's fast path for the 8-bit operators, is built with g++ against the
installed torch into ``dense_fp32_gemm_row_gb300/_tensors`` with this Python's suffix
for extension modules, and names that torch's version; the binding works without it,
so a torch it cannot be built for is only reported.
"""

from __future__ import annotations

import argparse
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgemmf32.so")
TENSORS_SRC = os.path.join(CSRC, "binding", "tensors.cpp")
TENSORS = os.path.join(PKG, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))
TENSORS_FOR = os.path.join(BUILD, "tensors.txt")  # the torch that TENSORS was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgemmf32.so")


def _sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers() -> list[str]:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(nvcc: str, src: str, force: bool) -> str:
    name = os.path.splitext(os.path.basename(src))[0]
    obj = os.path.join(BUILD, name + ".o")
    if not force and not _stale(obj, [src, *_headers(), __file__]):
        return obj
    cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xptxas", "-v", "-I", INCLUDE, "-c", src, "-o", obj + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(BUILD, name + ".ptxas.txt"), "w") as f:
        f.write(res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr[-4000:]}")
    os.replace(obj + ".tmp", obj)
    return obj


def _torch_version(torch_dir: str) -> str:
    """``torch.__version__`` of the torch in a folder, without importing it; "" if there is none."""
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            found = re.search(r"^__version__ = ['\"]([\w.+-]+)['\"]", f.read(), re.M)
    except OSError:
        return ""
    return found.group(1) if found else ""


def _build_tensors(force: bool) -> None:
    """Build the binding's module for the installed torch, if there is one.

    The module reads torch's objects by their layout in its headers, so one that was
    built for another torch is removed, whether or not it can be replaced.
    """
    import importlib.util

    spec = importlib.util.find_spec("torch")
    torch_dir = os.path.dirname(spec.origin) if spec is not None and spec.origin else ""
    version = _torch_version(torch_dir)
    made_for = f"{version} {torch_dir}"
    if not force and not _stale(TENSORS, [TENSORS_SRC, *_headers(), __file__]):
        if os.path.exists(TENSORS_FOR):
            with open(TENSORS_FOR) as f:
                if f.read() == made_for:
                    return
    for old in (TENSORS, TENSORS_FOR, os.path.join(PKG, "_tensors.so")):
        if os.path.exists(old):
            os.remove(old)
    if not version:
        return
    include = os.path.join(torch_dir, "include")
    lib = os.path.join(torch_dir, "lib")
    tmp = TENSORS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=1",
           f'-DTENSORS_TORCH="{version}"', "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           TENSORS_SRC, "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        failed = res.stderr[-2000:] if res.returncode else ""
    except OSError as e:  # no g++
        failed = str(e)
    if not failed:
        os.replace(tmp, TENSORS)
        with open(TENSORS_FOR, "w") as f:
            f.write(made_for)
    else:
        print(f"{TENSORS} not built, every call of an 8-bit operator goes step by step in Python:\n{failed}",
              file=sys.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build (if stale) and return the path of libgemmf32.so."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    with ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        tensors = ex.submit(_build_tensors, force)
        objs = list(ex.map(lambda s: _compile(nvcc, s, force), srcs))
        tensors.result()
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr[-4000:]}")
        os.replace(tmp, LIB)
    if verbose:
        for s in srcs:
            name = os.path.splitext(os.path.basename(s))[0]
            with open(os.path.join(BUILD, name + ".ptxas.txt")) as f:
                print(f"== {name}\n{f.read()}")
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
