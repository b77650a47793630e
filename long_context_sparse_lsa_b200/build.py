"""Build liblsa.so (the C-ABI library) from csrc/*.cu for sm_100a, and
_marshal.so (compiled argument handling of binding.py) from csrc/marshal.cpp.

Usage: python -m long_context_sparse_lsa_b200.build [--force] [--verbose]
Both are written next to this file (in-tree) so they travel with the
source tree; nvcc cross-compiles without a GPU.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "liblsa.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    out = []
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if f.endswith((".cu", ".cuh", ".h", ".cpp")):
                out.append(os.path.join(d, f))
    return out


def up_to_date() -> bool:
    if not (os.path.exists(LIBRARY) and os.path.exists(MARSHAL)):
        return False
    t = min(os.path.getmtime(LIBRARY), os.path.getmtime(MARSHAL))
    if any(os.path.getmtime(f) > t for f in _deps() + [os.path.abspath(__file__)]):
        return False
    with open(MARSHAL, "rb") as f:
        return built_for().encode() + b"\0" in f.read()


def built_for() -> str:
    """What _marshal.so is compiled against. It holds this text; another Python or torch cannot use it."""
    import torch

    return f"{sysconfig.get_config_var('SOABI')}, torch {torch.__version__}"


def _build_marshal(nvcc: str, verbose: bool) -> None:
    """_marshal.so, against the headers and libraries of the installed torch (which the importing process has loaded)."""
    import torch

    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
           sysconfig.get_paths()["include"], INCLUDE, BUILD_DIR]
    with open(os.path.join(BUILD_DIR, "built_for.h"), "w") as f:
        f.write(f'#define LSA_BUILT_FOR "{built_for()}"\n')
    tmp = MARSHAL + ".tmp"
    cmd = [nvcc, "-O2", "-shared", "-std=c++17", "-cudart", "none", "-Xcompiler", "-fPIC",  # (nvcc's host compiler)
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *["-I" + d for d in inc], os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L" + os.path.join(base, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("marshal.cpp, which the 4-bit and whole-prompt calls need, did not build (the library did):\n"
                           f"{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIBRARY
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + (extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        marshal = ex.submit(_build_marshal, nvcc, verbose)
        objs = list(ex.map(compile_one, sources()))
    tmp = LIBRARY + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    marshal.result()  # the library stands, and its other calls, where this one fails
    return LIBRARY


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print register/smem usage (-Xptxas -v)")
    args = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if args.ptxas_info else None
    print(build(force=args.force or args.ptxas_info, verbose=args.verbose or args.ptxas_info, extra=extra))
    return 0


if __name__ == "__main__":
    sys.exit(main())
