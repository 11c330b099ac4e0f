"""Build the KDA CUDA library and its Python binding in-tree for sm_103a (no cmake, no setuptools).

``python -m linear_attention_serving_chunkwise_gb300.build`` or ``build()`` compiles each
``csrc/*.cu`` translation unit in parallel with nvcc and links ``libkda_gb300.so`` beside this file, and ``_bind.so``, the
compiled part of the Python binding (``csrc/kda_bind.cpp``, with g++ and the installed PyTorch's headers).  Where there is no PyTorch,
``python build.py`` builds the library alone.
``build(phase_clocks=True)`` builds a separate instrumented library,
``libkda_gb300_clocks.so``, with the per-phase cycle marks compiled in (see phase_clocks.py);
the library everything else loads never has them.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda_gb300.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_SRC = os.path.join(CSRC, "kda_bind.cpp")
OBJ_CLOCKS = os.path.join(PKG, "_build_clocks")
LIB_CLOCKS = os.path.join(PKG, "libkda_gb300_clocks.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA library needs the CUDA 13 toolkit to build")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(os.path.dirname(PKG), "include", "kda.h")]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _has_torch() -> bool:
    if importlib.util.find_spec("torch"):
        return True
    sys.stderr.write("PyTorch is not installed: the C library is built without its Python binding\n")
    return False


def _bound_to() -> str:
    """What the binding is compiled for: this PyTorch, where it lies (a search path of the binding), and this Python."""
    import sysconfig
    import torch
    return "\n".join([torch.__version__, os.path.dirname(torch.__file__), str(sysconfig.get_config_var("SOABI"))])


def bind_up_to_date() -> bool:
    """Newer than its sources, and built for the PyTorch and the Python that run."""
    stamp = os.path.join(OBJ, "bind.torch")
    if not os.path.exists(BIND) or not os.path.exists(stamp) or open(stamp).read() != _bound_to():
        return False
    return all(os.path.getmtime(p) <= os.path.getmtime(BIND) for p in _deps() + [BIND_SRC])


def _compile_bind() -> str:
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    obj = os.path.join(OBJ, "kda_bind.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for i in includes:
        cmd += ["-isystem", i]
    r = subprocess.run(cmd + ["-c", BIND_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed on kda_bind.cpp")
    return obj


def _link_bind(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-shared", obj, "-o", BIND + ".tmp", "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L", libs,
           f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking _bind.so failed")
    os.replace(BIND + ".tmp", BIND)
    with open(os.path.join(OBJ, "bind.torch"), "w") as f:
        f.write(_bound_to())


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False, phase_clocks: bool = False) -> str:
    lib_path, obj_dir = (LIB_CLOCKS, OBJ_CLOCKS) if phase_clocks else (LIB, OBJ)
    current = not force and up_to_date(lib_path)
    bind = not phase_clocks and _has_torch() and (force or not current or not bind_up_to_date())
    if current and not bind:
        return lib_path
    os.makedirs(obj_dir, exist_ok=True)
    if current:
        _link_bind(_compile_bind())
        return lib_path
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "--expt-relaxed-constexpr", "-I", os.path.join(os.path.dirname(PKG), "include")]
    if phase_clocks:
        common += ["-DKDA_PHASE_CLOCKS"]
    if ptxas_v:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + common + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose or ptxas_v:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(_sources()))) as ex:
        bind_obj = ex.submit(_compile_bind) if bind else None
        objs = list(ex.map(compile_one, _sources()))
    libdir = _cuda_lib_dir(nvcc)
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", lib_path + ".tmp"] + objs + \
        ["-Xlinker", f"-rpath,{libdir}", "-L", libdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"linking {os.path.basename(lib_path)} failed")
    os.replace(lib_path + ".tmp", lib_path)
    if bind:
        _link_bind(bind_obj.result())
    return lib_path


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_v="--ptxas-v" in sys.argv)
    print(LIB)
