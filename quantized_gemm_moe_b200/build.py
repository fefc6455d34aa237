"""Builds the sm_100a CUDA library libqe.so in-tree (no JIT cache).

    python -m quantized_gemm_moe_b200.build [--force]

Every .cu under csrc/ is compiled with nvcc for sm_100a and linked into one
shared library next to this file. The C ABI is declared in include/qe.h.
csrc/qe_torch.cpp, the binding of the norm and MXFP4 operators for torch
tensors, becomes the extension module _qe_torch.so beside it.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libqe.so")
BINDING_SRC = os.path.join(CSRC, "qe_torch.cpp")
BINDING = os.path.join(HERE, "_qe_torch.so")
BINDING_ABI = os.path.join(HERE, "_build", "qe_torch.abi")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "qe.h")]


def _newer(out: str, inputs: list[str]) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _binding_abi() -> str:
    """What the module's binary interface hangs on: it calls torch's C++ and Python's C interface."""
    import sysconfig
    import torch
    return f"torch {torch.__version__} cxx11 {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}\n"


def binding_up_to_date() -> bool:
    """Newer than its sources, and built for the torch and the Python that would load it."""
    if not _newer(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "qe.h")]) or not os.path.exists(BINDING_ABI):
        return False
    with open(BINDING_ABI) as f:
        return f.read() == _binding_abi()


def build_binding(force: bool = False) -> str:
    """g++ against torch's headers; libqe.so is found next to the module."""
    if not force and binding_up_to_date():
        return BINDING
    import sysconfig
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", BINDING_SRC, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(t, "include"), "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
           "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L" + HERE, "-l:libqe.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        sys.stdout.write(r.stdout.decode(errors="replace"))
        raise RuntimeError("g++ failed for " + BINDING_SRC)
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_ABI), exist_ok=True)
    with open(BINDING_ABI, "w") as f:
        f.write(_binding_abi())
    return BINDING


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        build_binding()
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                    "-I" + os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"] + (extra or [])
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc()] + flags + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stdout.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp"
    subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-ldl", "-lrt", "-lpthread"],
                   check=True)
    os.replace(tmp, LIB)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
