"""Build libpdssm.so (the sm_100a CUDA kernels behind the C ABI) in-tree, and
_blocks.so (the native half of the block operators' binding).

    python -m structured_sparse_state_b200.build [--force] [--verbose]

nvcc compiles every csrc/*.cu for sm_100a only (no PTX fallback, no fast
math: denormals and IEEE division stay as written), one object per file in
parallel (under _build/), and links them into one shared library with the
CUDA runtime linked statically.  g++ compiles csrc/blocks_py.cpp against
torch's headers; it calls the C ABI and holds no arithmetic.
"""
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpdssm.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BINDING = os.path.join(HERE, "_blocks.so")
BINDING_SRC = os.path.join(CSRC, "blocks_py.cpp")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-O2",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]
OBJ_DIR = os.path.join(HERE, "_build")


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [
        os.path.join(INCLUDE, "pdssm.h"), __file__]
    return any(os.path.getmtime(f) > t for f in deps)


def build_binding(force: bool = False) -> str:
    """Compiles the native binding against torch's headers; it finds
    libpdssm.so beside itself."""
    deps = [BINDING_SRC, os.path.join(INCLUDE, "pdssm.h"), __file__]
    if not force and os.path.exists(BINDING) and \
            all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in deps):
        return BINDING
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
           os.path.join(cuda, "include")]
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-DTORCH_API_INCLUDE_EXTENSION_H", "-DTORCH_EXTENSION_NAME=_blocks",
        *[f"-isystem{d}" for d in inc], BINDING_SRC, "-o", BINDING + ".tmp",
        "-L" + HERE, "-l:" + os.path.basename(LIB), "-L" + tlib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
        "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + tlib])
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles every csrc/*.cu to an object (in parallel), then links the
    shared library, then the binding."""
    if not force and not _stale():
        build_binding()
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd[1:1] = ["-Xptxas", "-v"]
        subprocess.check_call(cmd)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, srcs))
    subprocess.check_call([nvcc, *LINK_FLAGS, "-o", LIB + ".tmp", *objs])
    os.replace(LIB + ".tmp", LIB)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
