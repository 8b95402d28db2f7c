"""Build libkvq.so in-tree for sm_100a with nvcc, and _calls.so against torch.

    python sm_b200/build.py [--force] [--verbose]

Every ``csrc/*.cu`` file compiles to an object under ``_build/`` (in
parallel), and the objects link into ``sm_b200/libkvq.so``;
``csrc/torch_calls.cpp`` (the paged calls of the Python binding) compiles with
the host compiler against torch's headers and libkvq.so into
``sm_b200/_calls.so``.  A source or header newer than its library triggers a
rebuild.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libkvq.so")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS_STAMP = os.path.join(BUILD, "calls.stamp")         # what _calls.so was built against
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _calls_against() -> str:
    import torch
    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, python {sys.version_info[:2]}"


def stamp_calls() -> None:
    os.makedirs(os.path.dirname(CALLS_STAMP), exist_ok=True)
    with open(CALLS_STAMP, "w") as f:
        f.write(_calls_against())


def calls_up_to_date() -> bool:
    deps = [CALLS_SRC, os.path.abspath(__file__), *glob.glob(os.path.join(ROOT, "include", "*.h"))]
    if not (os.path.exists(CALLS) and os.path.exists(CALLS_STAMP)):
        return False
    with open(CALLS_STAMP) as f:
        same = f.read() == _calls_against()
    return same and all(os.path.getmtime(p) <= os.path.getmtime(CALLS) for p in deps)


def build_calls(force: bool = False) -> str:
    if not force and calls_up_to_date():
        return CALLS
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = CALLS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for p in inc for a in ("-isystem", p)], CALLS_SRC, "-o", tmp, "-L", HERE, "-l:libkvq.so",
           "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {CALLS_SRC}:\n{res.stderr}")
    os.replace(tmp, CALLS)
    stamp_calls()
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        build_calls(force)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    build_calls(force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(args.force, args.verbose))
