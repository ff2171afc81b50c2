"""Build libqar.so in-tree with hipcc for gfx950, and the extension that
calls it from torch (_qar_torch.so, host code only).

Flags: -O3; -ffp-contract=off (no fused multiply-add unless written
explicitly); correctly rounded binary32 division; fp32 denormals kept (no
flush-to-zero flag); packed-fp32 instructions disabled."""
from __future__ import annotations

import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(HERE, "libqar.so")
EXTENSION = os.path.join(HERE, "_qar_torch.so")
SOURCES = [os.path.join(CSRC, name) for name in ("qar_kernels.hip", "qar_kv8.hip", "qar_kv8_pages.hip", "qar_kv8_shared.hip",
                                               "qar_mx4.hip", "qar_rotate.hip", "qar_api.cpp")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def build(output: str = LIBRARY, extra: list[str] | None = None, verbose: bool = False) -> str:
    """Compile every source (at once, they share nothing but headers) and
    link the shared library; returns its path."""
    tmp = output + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    def compile_one(source):
        obj = f"{output}.{os.path.basename(source)}.o"
        run([HIPCC, *FLAGS, *(extra or []), "-c", source, "-o", obj])
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = list(pool.map(compile_one, SOURCES))
    run([HIPCC, f"--offload-arch={ARCH}", *(extra or []), "-shared", *objects, "-o", tmp])
    for obj in objects:
        os.remove(obj)
    os.replace(tmp, output)
    return output


def build_extension(output: str = EXTENSION, verbose: bool = False) -> str:
    """Compile the extension against torch's headers and the libqar.so beside
    it, which it finds there when loaded; returns its path."""
    import torch
    home = os.path.dirname(torch.__file__)
    includes = [INCLUDE] + [a for d in (os.path.join(home, "include"),
                                        os.path.join(home, "include", "torch", "csrc", "api", "include"),
                                        os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
                                        sysconfig.get_paths()["include"]) for a in ("-isystem", d)]
    tmp = output + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", *includes,
           os.path.join(CSRC, "qar_torch.cpp"), "-o", tmp, f"-L{HERE}", "-l:libqar.so", f"-L{os.path.join(home, 'lib')}",
           "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, output)
    return output


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_extension(verbose=True))
