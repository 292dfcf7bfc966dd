"""Build libentro.so in-tree with nvcc for sm_100a (B200), and the Python binding's extension module (_binding.so).

    python huffman_decode_canonical_b200/build.py [--verbose-ptxas]

(Run it as a script: importing the package itself loads libentro.so.)

The shared library lands next to this file, so it travels with the source
tree.  Host code is compiled without floating-point contraction so that the
encoder's quantization is reproducible bit for bit.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libentro.so")
OBJECTS = os.path.join(HERE, "_build")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_MADE_FOR = os.path.join(OBJECTS, "binding_made_for.txt")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("decode.cu", "product.cu", "prompt.cu", "kvcache.cu", "encoder.cpp", "launch.cpp")]
HEADERS = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))) + [
    os.path.join(ROOT, "include", "entro.h")]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _stale(target: str, sources) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in sources)


def _object(src: str) -> str:
    return os.path.join(OBJECTS, os.path.basename(src) + ".o")


def _binding_command(target: str):
    """The extension module over torch's tensors (host code only)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    includes = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include")] + cpp_extension.include_paths("cuda")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *[f"-I{p}" for p in includes], BINDING_SOURCE, "-o", target, f"-L{libs}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch",
            "-lc10_cuda", "-lc10"]


def _binding_wanted() -> bool:
    """A build of torch without CUDA has nothing to link the module with, and no tensors to call it with."""
    import torch
    return torch.version.cuda is not None


def _binding_abi() -> str:
    """What the module is bound to besides its source: torch's C++ interface and the interpreter's."""
    import sysconfig

    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _binding_stale() -> bool:
    try:
        with open(BINDING_MADE_FOR) as f:
            made_for = f.read()
    except FileNotFoundError:
        return True
    return made_for != _binding_abi() or _stale(BINDING, [BINDING_SOURCE, os.path.join(ROOT, "include", "entro.h")])


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    lib, binding = force or _stale(LIB, SOURCES + HEADERS), _binding_wanted() and (force or _binding_stale())
    if not lib and not binding:
        return LIB
    os.makedirs(OBJECTS, exist_ok=True)
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
             "-Xcompiler", "-fPIC,-pthread,-ffp-contract=off,-fvisibility=hidden",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if verbose_ptxas:
        flags = ["-Xptxas", "-v"] + flags
    running = []
    for src in SOURCES:  # the sources side by side
        if lib and (force or _stale(_object(src), [src] + HEADERS)):
            tmp = _object(src) + f".tmp{os.getpid()}"
            cmd = [NVCC] + flags + ["-c", "-o", tmp, src]
            running.append((cmd, tmp, _object(src), subprocess.Popen(cmd)))
    if binding:
        tmp = BINDING + f".tmp{os.getpid()}"
        cmd = _binding_command(tmp)
        running.append((cmd, tmp, BINDING, subprocess.Popen(cmd)))
    bad = None
    for cmd, tmp, obj, p in running:
        if p.wait() != 0:
            bad = bad or (p.returncode, cmd)
        else:
            os.replace(tmp, obj)
            if obj == BINDING:
                with open(BINDING_MADE_FOR, "w") as f:
                    f.write(_binding_abi())
    if bad:
        raise subprocess.CalledProcessError(*bad)
    if not lib:
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp]
                          + [_object(s) for s in SOURCES] + ["-lpthread"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv)
    print(LIB)
