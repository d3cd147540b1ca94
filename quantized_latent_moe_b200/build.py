"""Build libelq.so (the C ABI of include/elq.h and include/elq_ops.h) in-tree with nvcc for
sm_100a, and _ops.so, the compiled Python binding of the latter, with the host compiler."""
from __future__ import annotations

import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = [os.path.join(HERE, d) for d in ("csrc", "csrc_ops")]
OBJ = os.path.join(HERE, "_build")          # one object per source, rebuilt when stale
LIB = os.path.join(HERE, "libelq.so")
BINDING = os.path.join(HERE, "_ops.so")
BINDING_SRC = os.path.join(CSRC[1], "ops_binding.cpp")
BINDING_FOR = os.path.join(OBJ, "_ops.for")     # what _ops.so was built against
CXX = os.environ.get("CXX", "g++")
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
        raise RuntimeError("the compiler failed building libelq.so or _ops.so")
    return "".join(outs)


def _stale(target, sources):
    return not os.path.exists(target) or os.path.getmtime(target) < max(os.path.getmtime(p) for p in sources)


def binding_abi():
    """_ops.so holds for one Python and one torch; another of either needs another build."""
    return "%s torch %s" % (sys.implementation.cache_tag, importlib.metadata.version("torch"))


def _binding_stale():
    if _stale(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "elq.h"), os.path.join(ROOT, "include", "elq_ops.h"),
                        __file__]):
        return True
    try:
        with open(BINDING_FOR) as f:
            return f.read() != binding_abi()
    except OSError:
        return True


def _binding_cmd(out):
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
            *["-I" + p for p in inc], BINDING_SRC, "-o", out, "-L" + HERE, "-l:libelq.so",
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python",
            "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    out = ""
    if force or extra or _stale(LIB, deps()):
        os.makedirs(OBJ, exist_ok=True)
        cmds, objs, done = [], [], []
        for src in sources():
            obj = os.path.join(OBJ, os.path.basename(src) + ".o")
            objs.append(obj)
            if force or extra or _stale(obj, [src] + headers(src)):
                tmp = obj + ".tmp%d" % os.getpid()
                cmds.append([NVCC, *(["-Xptxas=-v"] if verbose else []), *FLAGS, *extra, "-c", "-o", tmp, src])
                done.append((tmp, obj))
        out = _run(cmds)
        for tmp, obj in done:
            os.replace(tmp, obj)
        tmp = LIB + ".tmp%d" % os.getpid()
        out += _run([[NVCC, *FLAGS, "-shared", "-o", tmp, *objs]])
        os.replace(tmp, LIB)
    if force or _binding_stale():
        os.makedirs(OBJ, exist_ok=True)
        tmp = BINDING + ".tmp%d" % os.getpid()
        out += _run([_binding_cmd(tmp)])
        os.replace(tmp, BINDING)
        with open(BINDING_FOR + ".tmp%d" % os.getpid(), "w") as f:
            f.write(binding_abi())
        os.replace(f.name, BINDING_FOR)
    if verbose:
        sys.stderr.write(out)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
