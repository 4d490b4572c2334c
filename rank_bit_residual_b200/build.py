"""Build libsvdq.so in-tree with nvcc for sm_100a.

    python -m rank_bit_residual_b200.build [--force]

Each csrc/*.cu file is compiled separately (in parallel) into _build/ and the
objects are linked into rank_bit_residual_b200/libsvdq.so. The CUDA runtime is
linked statically; the driver API is reached through cudaGetDriverEntryPoint,
so loading the library needs no libcuda at link time. csrc/attention_calls.cpp, the
quick calls of the attention operators, is compiled against torch and Python with the host
compiler and becomes rank_bit_residual_b200/_calls.<Python's ABI>.torch-<version>.so: it reads torch's
own types, so another Python or torch looks for another file and never takes this one.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsvdq.so")
CALLS_SRC = os.path.join(CSRC, "attention_calls.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I" + INCLUDE,
         "--expt-relaxed-constexpr", "-diag-suppress", "128,177"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libsvdq.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def calls_path() -> str:
    """Where the quick calls for this Python and this torch are."""
    import torch
    abi = f"{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}"
    if not torch.compiled_with_cxx11_abi():
        abi += "-oldabi"
    return os.path.join(PKG, f"_calls.{abi}.so")


def calls_up_to_date() -> bool:
    path = calls_path()
    deps = [CALLS_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def calls_command(out: str):
    """The host compiler's command line for the quick calls."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    lib = os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I" + INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], CALLS_SRC, "-o", out,
            "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _start_calls(force: bool):
    """The compiler of the quick calls at work, why it cannot be, or None: nothing to do."""
    try:
        if not force and calls_up_to_date():
            return None
        return subprocess.Popen(calls_command(calls_path() + ".tmp"), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except (ImportError, OSError, RuntimeError) as e:   # no torch, no g++, no CUDA headers
        return str(e)


def _finish_calls(calls) -> None:
    """The library is complete without the quick calls, so a failure is a warning."""
    if not isinstance(calls, str):
        out, _ = calls.communicate()
        if calls.returncode == 0:
            os.replace(calls_path() + ".tmp", calls_path())
            return
        calls = out.decode(errors="replace")
    warnings.warn(f"the quick calls of the attention operators were not built, the calls without them are:\n{calls}",
                  RuntimeWarning, stacklevel=3)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path. Raises if the library cannot be built, and
    warns if only the quick calls cannot."""
    calls = _start_calls(force)
    try:
        if force or not up_to_date():
            _build_library(verbose)
    finally:
        if calls is not None:
            _finish_calls(calls)
    return LIB


def _build_library(verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"))
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(path)
