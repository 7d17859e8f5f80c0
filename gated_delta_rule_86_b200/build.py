"""In-tree build of the CUDA library (nvcc, sm_100a).

``build_library()`` compiles ``csrc/kda_api.cu`` (which includes every kernel)
into ``libkda_b200.so`` next to this file.  The build is skipped when the
library is newer than every source file.  ``build_binding()`` compiles the native
binding of the attention calls against torch's headers.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libkda_b200.so")
BINDING_PATH = os.path.join(HERE, "_attention.so")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH_FLAGS + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda_b200.so")


def _sources():
    return (glob.glob(os.path.join(HERE, "csrc", "*.cu")) + glob.glob(os.path.join(HERE, "csrc", "*.cuh"))
            + [os.path.join(ROOT, "include", "kda.h")])


def _stale(target, sources):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def compile_so(src: str, out: str, deps, extra=(), force=False) -> str:
    if force or _stale(out, list(deps) + [src]):
        tmp = out + f".tmp{os.getpid()}"
        cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-o", tmp, src]
        subprocess.check_call(cmd)
        os.replace(tmp, out)
    return out


def build_library(force: bool = False) -> str:
    return compile_so(os.path.join(HERE, "csrc", "kda_api.cu"), LIB_PATH, _sources(), force=force)


def build_binding(force: bool = False) -> str:
    """The native Python binding of the attention calls (g++, torch's headers), beside the library that it
    links to."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    src = os.path.join(HERE, "csrc", "attn_binding.cpp")
    made_for = f"built for torch {torch.__version__}"   # it uses torch's internals, which change between versions

    def other_torch():
        with open(BINDING_PATH, "rb") as f:
            return made_for.encode() + b"\0" not in f.read()

    if not (force or _stale(BINDING_PATH, [src, os.path.join(ROOT, "include", "kda.h")]) or other_torch()):
        return BINDING_PATH
    build_library()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DTORCH_API_INCLUDE_EXTENSION_H",
           "-DTORCH_EXTENSION_NAME=_attention", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DKDA_BUILT_FOR="{made_for}"']
    for d in include_paths() + [os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += [src, "-o", tmp, f"-L{libs}", f"-L{HERE}", "-l:libkda_b200.so", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build_probe(force: bool = False) -> str:
    """Test-only probe libraries (tests/csrc): tcgen05 layouts, and parts of the attention kernels."""
    for name in ("attn_probe", "tc_probe"):
        out = compile_so(os.path.join(ROOT, "tests", "csrc", f"{name}.cu"), os.path.join(ROOT, "tests", "csrc", f"lib{name}.so"),
                         _sources(), force=force)
    return out


if __name__ == "__main__":
    print(build_library(force=True))
    print(build_binding(force=True))
    print(build_probe(force=True))
