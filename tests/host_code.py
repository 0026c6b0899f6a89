"""Functions of the kernels' headers that also compile for the host, built into
a library of their own for a test: what a block computes from its number, checked
without a GPU."""
import ctypes
import os
import subprocess

from shared_memory_tiled_amd import build


def compile_host(tmp_path, source, overflow="-fwrapv"):
    """The C functions of ``source`` (HIP, host side only) as a ctypes library;
    ``overflow``: what a signed one does."""
    src, lib = os.path.join(tmp_path, "host.hip"), os.path.join(tmp_path, "host.so")
    with open(src, "w") as f:
        f.write(source)
    # by default it wraps, and shows as the wrong place that it gives
    cmd = [build.HIPCC, "--cuda-host-only", "-O1", "-std=c++17", overflow, "-fPIC", "-shared", "-w", "-I", build.INCLUDE,
           "-I", build.CSRC, src, "-o", lib]
    subprocess.run(cmd, check=True)
    return ctypes.CDLL(lib)
