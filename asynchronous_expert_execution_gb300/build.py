"""Build the in-tree shared libraries for sm_103a.

``libmoe_async.so`` is the release library; ``libmoe_async_debug.so`` is the same code
compiled with MOE_DEBUG_BOUNDS, which checks every bucket, slot and k index the kernels read
back from device state and latches MOE_ERR_BOUNDS instead of touching memory out of range
(loaded when the environment sets MOE_DEBUG_BOUNDS=1).  nvcc compiles every translation unit
of both under ``csrc/`` in parallel and links each set into one shared object next to this
file.  ``_ops.so`` is the Python binding of the stateless operators (g++ against torch, no
device code; it calls whichever library was loaded).  A rebuild is skipped when a library is
newer than every source and header, and the binding was built for the torch and Python at hand.
"""
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmoe_async.so")
LIB_DEBUG = os.path.join(HERE, "libmoe_async_debug.so")
BINDING = os.path.join(HERE, "_ops.so")
BINDING_SRC = os.path.join(CSRC, "moe_binding.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")
BINDING_TAG = os.path.join(BUILD_DIR, "binding.tag")
VARIANTS = {"release": (LIB, []), "debug": (LIB_DEBUG, ["-DMOE_DEBUG_BOUNDS=1"])}

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE]
# The tcgen05 kernels must not spill: one holds an SM's whole register file, and a build of a
# variant that spilled faulted on the GPU.  ptxas turns a spill into a build error.
FILE_FLAGS = {f: ["-Xptxas", "--warn-on-spills,--warning-as-error"] for f in ("moe_ffn_tc.cu", "moe_linear.cu", "moe_linear_backward.cu", "moe_linear_blocks.cu")}


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_async.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [BINDING_SRC]
    return any(os.path.getmtime(p) > t for p in deps)


def binding_tag():
    """What the binding is built against: it uses torch's C++ classes, whose layout changes between versions."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"


def _binding_stale():
    if _stale(BINDING) or not os.path.exists(BINDING_TAG):
        return True
    with open(BINDING_TAG) as f:
        return f.read() != binding_tag()


def _binding_cmd(out):
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [x for p in cpp_extension.include_paths("cuda") for x in ("-isystem", p)]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DMOE_BINDING_TAG="{binding_tag()}"',
            *inc, "-I", sysconfig.get_paths()["include"], BINDING_SRC, "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def build(force=False, verbose=False, variants=("release", "debug")):
    """Compile and link the requested libraries (all translation units of all of them in
    parallel); returns the release library's path."""
    todo = [v for v in variants if force or _stale(VARIANTS[v][0])]
    binding = force or _binding_stale()
    if not todo and not binding:
        return LIB
    procs, objs = [], {}
    if binding:
        os.makedirs(BUILD_DIR, exist_ok=True)
        cmd = _binding_cmd(BINDING + ".tmp")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((BINDING_SRC, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    nvcc = _nvcc() if todo else None
    for v in todo:
        bdir = os.path.join(BUILD_DIR, v)
        os.makedirs(bdir, exist_ok=True)
        objs[v] = []
        for src in sources():
            obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, *FILE_FLAGS.get(os.path.basename(src), []), *VARIANTS[v][1],
                   "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
            objs[v].append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    if binding:
        os.replace(BINDING + ".tmp", BINDING)
        with open(BINDING_TAG, "w") as f:
            f.write(binding_tag())
    for v in todo:
        lib = VARIANTS[v][0]
        tmp = lib + ".tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs[v]]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
