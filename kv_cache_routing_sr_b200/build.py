"""Builds libsinkrouter.so in-tree with nvcc for sm_100a.

    python -m kv_cache_routing_sr_b200.build [--verbose-ptxas] [-DNAME=VALUE ...]

The library is the C ABI declared in include/sinkrouter.h. cudart is linked
statically, so the .so needs only the NVIDIA driver at run time. Beside it goes
_sr_binding.so (g++, against the installed torch), which the Python package uses to
check tensors and call the library.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libsinkrouter.so")
BINDING = os.path.join(PKG, "_sr_binding.so")
SOURCES = ["sr_abi.cu", "sr_route.cu", "sr_prestep.cu", "sr_decode.cu", "sr_combine.cu", "sr_static_scratch.cu",
           "sr_selftest.cu", "sr_position0.cu", "sr_kv_quant.cu", "sr_prefix.cu", "sr_tensormap.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libsinkrouter.so")
    return cand


def _run(cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _binding_mark() -> bytes:
    """What a binding compiled against the installed torch contains."""
    import torch
    return f"sr_binding for torch {torch.__version__};".encode()


def binding_current(path: str = BINDING) -> bool:
    """Whether the Python binding is there and was compiled against the installed torch
    (its C++ interface is fixed within one version only)."""
    if not os.path.exists(path):
        return False
    with open(path, "rb") as f:
        return _binding_mark() in f.read()


def build_binding(output: str = BINDING) -> str:
    """Compile the Python binding against the installed torch and return its path."""
    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    lib = os.path.join(root, "lib")
    tmp = f"{output}.{os.getpid()}.tmp"
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f'-DSR_BINDING_MARK="{_binding_mark().decode()}"', *[f"-I{i}" for i in inc],
          os.path.join(CSRC, "sr_binding.cpp"), "-o", tmp, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
          "-ltorch_python", f"-Wl,-rpath,{lib}"])
    os.replace(tmp, output)
    return output


def build(output: str = LIBRARY, defines=(), verbose_ptxas: bool = False, quiet: bool = True) -> str:
    """Compile every source into ``output`` (a shared library) and return its path.
    The in-tree library brings the Python binding with it."""
    flags = [*ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}",
             *[f"-D{d}" for d in defines]]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    tmp = f"{output}.{os.getpid()}.tmp"
    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor(len(SOURCES) + 1) as pool:
        binding = pool.submit(build_binding) if os.path.abspath(output) == os.path.abspath(LIBRARY) else None
        objs = [os.path.join(objects, s + ".o") for s in SOURCES]  # one compiler a source, side by side
        said = list(pool.map(_run, [[nvcc(), *flags, "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objs)]))
        said.append(_run([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "--cudart", "static", *objs, "-o", tmp]))
        if binding is not None:
            binding.result()
    if not quiet or verbose_ptxas:
        sys.stderr.write("".join(said))
    os.replace(tmp, output)
    return output


def needs_build(output: str = LIBRARY) -> bool:
    if not os.path.exists(output) or not binding_current():
        return True
    newest = max(os.path.getmtime(os.path.join(CSRC, f)) for f in os.listdir(CSRC))
    newest = max(newest, os.path.getmtime(os.path.join(INCLUDE, "sinkrouter.h")))
    return min(os.path.getmtime(output), os.path.getmtime(BINDING)) < newest


if __name__ == "__main__":
    args = sys.argv[1:]
    defs = [a[2:] for a in args if a.startswith("-D")]
    print(build(defines=defs, verbose_ptxas="--verbose-ptxas" in args, quiet=False))
