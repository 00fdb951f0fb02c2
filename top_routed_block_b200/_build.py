"""Builds libfvattn.so in-tree with nvcc for sm_100a (no JIT cache, no torch extension), and beside
it the Python module _binding (host C++ against torch) for the calls that run for single tokens.

    python -m top_routed_block_b200._build
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libfvattn.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(PKG, "_build", "binding.txt")   # the Python and torch that BINDING was compiled against
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-diag-suppress", "1160"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(PKG, "csrc", "*.cuh")) + glob.glob(os.path.join(PKG, "csrc", "*.h")) + [os.path.join(ROOT, "include", "fvattn.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def _newer(paths, than: str) -> bool:
    return not os.path.exists(than) or any(os.path.getmtime(p) > os.path.getmtime(than) for p in paths)


def binding_target() -> str:
    """What the binding is compiled against: torch's C++ interface is another one in each release."""
    import torch
    return f"python {sys.version_info[0]}.{sys.version_info[1]}, torch {torch.__version__}"


def _binding_stale() -> bool:
    if _newer([os.path.join(PKG, "csrc", "binding.cpp"), os.path.join(ROOT, "include", "fvattn.h")], BINDING):
        return True
    if not os.path.exists(BUILT_FOR):
        return True
    with open(BUILT_FOR) as f:
        return f.read() != binding_target()


def _build_binding(force: bool) -> None:
    src = os.path.join(PKG, "csrc", "binding.cpp")
    if not force and not _binding_stale():
        return
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = BINDING + ".tmp"
    subprocess.check_call([
        "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        f'-DFVATTN_BUILT_FOR="{binding_target()}"',
        "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
        "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
        "-isystem", os.path.join(cuda, "include"), src, "-o", tmp, "-L", PKG, "-lfvattn", "-Wl,-rpath,$ORIGIN",
        "-L", lib, "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda"])
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BUILT_FOR), exist_ok=True)
    with open(BUILT_FOR, "w") as f:
        f.write(binding_target())


def build(force: bool = False, verbose: bool = False) -> str:
    lib = _build_library(force, verbose)
    _build_binding(force)
    return lib


def _build_library(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    failed = False
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stderr.write(out)
        failed |= p.returncode != 0
    if failed:
        raise RuntimeError("nvcc failed")
    tmp = LIB + ".tmp"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
