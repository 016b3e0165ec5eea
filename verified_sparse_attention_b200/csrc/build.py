"""Build libvattn.so (the C-ABI library) for sm_100a with nvcc, in-tree.

    python -m verified_sparse_attention_b200.csrc.build [--ptxas-verbose]
"""
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(HERE, f) for f in ("vattn_api.cu", "vattn_static.cu", "vattn_append.cu", "vattn_shared.cu")]
DEPS = [*SRCS, *(os.path.join(HERE, f) for f in ("vattn_kernels.cuh", "vattn_device.cuh", "vattn_ctx.h", "vattn_shared.cuh", "vattn_prefix_tc.cuh")),
        os.path.join(ROOT, "include", "vattn.h")]
OUT = os.path.join(PKG, "libvattn.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", HERE]


def needs_build():
    if not os.path.exists(OUT):
        return True
    t = os.path.getmtime(OUT)
    return any(os.path.getmtime(d) > t for d in DEPS)


def build(verbose_ptxas=False, out=OUT):
    """Compile every source (side by side) and link the library."""
    more = ["-Xptxas", "-v"] if verbose_ptxas else []
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SRCS]
        cmds = [[NVCC, *more, *FLAGS, "-c", s, "-o", o] for s, o in zip(SRCS, objs)]
        procs = [subprocess.Popen(c) for c in cmds]
        status = [p.wait() for p in procs]
        for c, rc in zip(cmds, status):
            if rc:
                raise subprocess.CalledProcessError(rc, c)
        subprocess.run([NVCC, *FLAGS, "-shared", *objs, "-o", out], check=True)
    return out


if __name__ == "__main__":
    print(build(verbose_ptxas="--ptxas-verbose" in sys.argv))
