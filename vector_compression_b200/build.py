"""Build libtq.so in-tree for sm_100a with nvcc.

    python -m vector_compression_b200.build [--force]

The shared library is written next to this file so that it travels with the
source tree, and with it _torch_binding.so, the calls on torch tensors that run
once per layer and step; both are rebuilt when any source under csrc/, binding/ or
include/ is newer.  Without torch the library alone is built, which a user of the
C ABI needs nothing but nvcc and its host compiler for.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import time

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtq.so")
# the calls on torch tensors, a Python module that is linked against libtq.so
BINDING_SRC = os.path.join(HERE, "binding", "tq_torch.cpp")
BINDING = os.path.join(HERE, "_torch_binding.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def needs_build() -> bool:
    built, of = ([LIB, BINDING], deps() + [BINDING_SRC]) if has_torch() else ([LIB], deps())
    if not all(os.path.exists(f) for f in built):
        return True
    t = min(os.path.getmtime(f) for f in built)
    return any(os.path.getmtime(f) > t for f in of)


def binding_commands(obj: str, out: str):
    """Compile and link commands of the binding (torch's headers and libraries, this interpreter's)."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-DTORCH_EXTENSION_NAME=_torch_binding",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *[x for i in inc for x in ("-isystem", i)], "-c", BINDING_SRC, "-o", obj]
    link = ["g++", "-shared", "-o", out, obj, "-L" + HERE, "-l:libtq.so", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    return compile_, link


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    t0 = time.time()
    procs = []
    objs = []
    link_binding = None
    if has_torch():
        compile_binding, link_binding = binding_commands(os.path.join(objdir, "tq_torch.cpp.o"), BINDING + ".tmp")
        procs.append((compile_binding, subprocess.Popen(compile_binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            sys.stderr.write(out.decode(errors="replace"))
            raise RuntimeError("compilation failed: " + " ".join(cmd))
        if verbose and out:
            sys.stderr.write(out.decode(errors="replace"))
    tmp = LIB + ".tmp"
    link = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
            "-lcudart"]
    subprocess.run(link, check=True)
    os.replace(tmp, LIB)
    if link_binding:
        subprocess.run(link_binding, check=True)
        os.replace(BINDING + ".tmp", BINDING)
    if verbose:
        print(f"built {LIB} in {time.time() - t0:.1f}s" + ("" if link_binding else " (no torch: without its binding)"))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
