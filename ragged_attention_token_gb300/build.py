"""Build librra.so (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc.

    python -m ragged_attention_token_gb300.build [--verbose] [--force] [--ptxas-info]

Each .cu file in csrc/ compiles to an object in parallel; the objects link
into ragged_attention_token_gb300/librra.so against the shared CUDA runtime.
csrc/fastcall.cpp becomes a Python extension beside it (fast_path()).  A rebuild happens only when a source or header is newer than the library.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "librra.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O3,-fvisibility=hidden", "-I", INCLUDE,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: librra.so cannot be built")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    deps += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    deps.append(os.path.abspath(__file__))
    return deps


# The block operators' argument marshalling in C++ (a Python extension against
# torch's headers).  Without it rra.py marshals those calls itself.
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")


def fast_path() -> str:
    """Where the extension for this torch and this Python lies: one built against another is another file, never loaded here."""
    import torch
    return os.path.join(PKG_DIR, f"_rra_fast-torch{torch.__version__}-{sys.implementation.cache_tag}.so")


def _fast_up_to_date() -> bool:
    path = fast_path()
    deps = [FAST_SRC, os.path.join(INCLUDE, "rra.h"), os.path.abspath(__file__)]
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def build_fast(verbose: bool = False, force: bool = False) -> str:
    """Compile the marshalling extension with the host compiler; returns its path."""
    path = fast_path()
    if not force and _fast_up_to_date():
        return path
    import sysconfig

    import torch
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(troot, "include"),
           os.path.join(troot, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = path + ".tmp"
    if os.path.exists(path):
        os.remove(path)                    # should the build fail, an extension of older sources is not to be used
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[x for d in inc for x in ("-isystem", d)],
          FAST_SRC, "-o", tmp, "-L", os.path.join(troot, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
         verbose)
    os.replace(tmp, path)
    return path


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _run(cmd: list[str], verbose: bool) -> str:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}")
    return r.stdout


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link librra.so; returns its path."""
    try:
        build_fast(verbose=verbose, force=force)
    except (RuntimeError, OSError, ImportError) as e:
        print(f"the marshalling extension was not built (calls are marshalled in Python): {e}", file=sys.stderr)
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        jobs.append((obj, [nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        outs = list(ex.map(lambda j: _run(j[1], verbose), jobs))
    if ptxas_info or verbose:
        for (obj, _), out in zip(jobs, outs):
            if out.strip():
                print(f"== {os.path.basename(obj)}\n{out}", flush=True)
    tmp = LIB_PATH + ".tmp"
    _run([nvcc, *ARCH_FLAGS, "-shared", "--cudart", "shared", "-o", tmp, *[o for o, _ in jobs]], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / smem per kernel")
    args = ap.parse_args(argv)
    path = build(verbose=args.verbose, force=args.force or args.ptxas_info, ptxas_info=args.ptxas_info)
    print(path)
    return 0


if __name__ == "__main__":
    sys.exit(main())
