"""Build libmxa.so in-tree for sm_100a.

    python -m decode_attention_packed_b200.build [--force] [--verbose]

nvcc cross-compiles without a GPU; the library links the CUDA runtime
statically and looks the tensor-map encoder up through the runtime's driver
entry point, so it loads on a machine without a GPU as well.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmxa.so")
# (source, object, its own flags): the split kernel's instances of each head
# dim are compiled apart, side by side
UNITS = [("mxa_kernels.cu", "mxa_kernels_d%d.o" % d, ["-DMXA_HEAD_DIM=%d" % d]) for d in (64, 128, 256)] + \
    [(f, f + ".o", []) for f in ("mxa_api.cpp", "mxa_noalloc.cu", "mxa_cache_ops.cu", "mxa_prefill.cu")]
DEPS = sorted({os.path.join(CSRC, u[0]) for u in UNITS}) + \
    [os.path.join(CSRC, f) for f in ("mxa_config.h", "mxa_device.cuh", "mxa_launch.h", "mxa_prefill.h",
                                    "mxa_tcgen05.cuh", "mxa_tmap.h")] + \
    [os.path.join(INCLUDE, "mxa.h")]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I" + INCLUDE, "-I" + CSRC]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in DEPS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    objs, running = [], []
    for src, obj, extra in UNITS:
        obj = os.path.join(CSRC, obj)
        cmd = [NVCC, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose and src.endswith(".cu"):
            cmd += ["-Xptxas", "-v"]
        running.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    failed = [subprocess.CalledProcessError(p.returncode, cmd) for cmd, p in running if p.wait() != 0]
    if failed:
        raise failed[0]
    tmp = LIB + ".tmp"
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                           "-Xcompiler", "-fPIC", *objs, "-o", tmp, "-lcudart_static", "-ldl", "-lrt",
                           "-lpthread"])
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
