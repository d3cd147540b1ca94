"""Build libelq.so (the C ABI of include/elq.h) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = [os.path.join(HERE, d) for d in ("csrc", "csrc_ops")]
OBJ = os.path.join(HERE, "_build")          # one object per source, rebuilt when stale
LIB = os.path.join(HERE, "libelq.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-fmad=false",            # no contraction: every fused multiply-add is explicit
    "-Xcompiler", "-fPIC",
    "-I" + os.path.join(ROOT, "include"),
]


def sources():
    return [p for d in CSRC for p in sorted(glob.glob(os.path.join(d, "*.cu")))]


def headers(src):
    """What an object of `src` depends on: its folder's headers, the device
    helpers that both folders share, and the C headers."""
    own = os.path.dirname(src)
    shared = sorted(glob.glob(os.path.join(CSRC[0], "*.cuh"))) if own == CSRC[0] else [
        os.path.join(CSRC[0], "elq_device.cuh")] + sorted(glob.glob(os.path.join(own, "*.cuh")))
    return shared + [os.path.join(ROOT, "include", "elq.h"), os.path.join(ROOT, "include", "elq_ops.h"), __file__]


def deps():
    return sorted({p for s in sources() for p in [s] + headers(s)})


def _run(cmds):
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
    outs = [p.communicate()[0] for p in procs]
    if any(p.returncode for p in procs):
        sys.stderr.write("".join(outs))
        raise RuntimeError("nvcc failed building libelq.so")
    return "".join(outs)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    newest = max(os.path.getmtime(p) for p in deps())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    cmds, objs, done = [], [], []
    for src in sources():
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or extra or not os.path.exists(obj) or os.path.getmtime(obj) < max(
                os.path.getmtime(p) for p in [src] + headers(src)):
            tmp = obj + ".tmp%d" % os.getpid()
            cmds.append([NVCC, *(["-Xptxas=-v"] if verbose else []), *FLAGS, *extra, "-c", "-o", tmp, src])
            done.append((tmp, obj))
    out = _run(cmds)
    for tmp, obj in done:
        os.replace(tmp, obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    out += _run([[NVCC, *FLAGS, "-shared", "-o", tmp, *objs]])
    if verbose:
        sys.stderr.write(out)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
