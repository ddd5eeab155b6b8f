"""Builds the in-tree CUDA libraries (sm_100a) with nvcc: ``libmoe_b200.so`` and
``libmoe_b200_debug.so``, the same sources compiled with MOE_DEBUG (the
checking build: table-dependent accesses are checked against their buffers
and flagged with MOE_DEVERR_BOUNDS); and with g++ the Python module that
marshals the short calls (``moe_binding.cpp``, host code against the installed
torch and Python, whose versions its file name carries)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_b200.so")
LIB_DEBUG = os.path.join(HERE, "libmoe_b200_debug.so")
SOURCES = ["moe_kernels.cu", "moe_api.cu", "moe_products.cu", "moe_noalloc.cu"]
HEADERS = ["moe_device.cuh", "moe_gemm.cuh", "moe_gemm_fp8.cuh", "moe_gemm2.cuh", "moe_gemm2_fp8.cuh", "moe_ragged.cuh", "moe_split.cuh",
           "moe_rows.cuh", "moe_host.h", "moe_launch.h", os.path.join("..", "..", "include", "moe.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


BINDING_SOURCE = os.path.join(CSRC, "moe_binding.cpp")


def binding_path() -> str:
    """One file for each torch and each interpreter: the module is built against the headers of both."""
    import sysconfig

    import torch
    version = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(HERE, f"_binding_{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_stale() -> bool:
    """Whether the marshalling module is missing or older than its sources."""
    path = binding_path()
    deps = [BINDING_SOURCE, os.path.join(HERE, "..", "include", "moe.h")]
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps if os.path.exists(p))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Builds the marshalling module when it is missing or older than its sources; returns its path."""
    import sysconfig

    import torch

    path = binding_path()
    if not force and not binding_stale():
        return path
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in inc], BINDING_SOURCE,
           "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)
    return path


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def _build_variants(variants, verbose: bool, ptxas_verbose: bool) -> None:
    """Compiles every (variant, source) object in parallel, then links each library."""
    jobs, variants_objs = [], []
    for lib, defines, sub in variants:
        build_dir = os.path.join(HERE, "_build", sub)
        os.makedirs(build_dir, exist_ok=True)
        objs = []
        for src in SOURCES:
            obj = os.path.join(build_dir, src.replace(".cu", ".o"))
            cmd = [_nvcc(), *NVCC_FLAGS, *defines, "-c", os.path.join(CSRC, src), "-o", obj]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            jobs.append((subprocess.Popen(cmd), cmd))
            objs.append(obj)
        variants_objs.append((lib, objs))
    failed = [cmd for proc, cmd in jobs if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for lib, objs in variants_objs:
        tmp = lib + f".tmp{os.getpid()}"
        subprocess.run([_nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", tmp,
                        "-lcudart", "-ldl"], check=True)
        os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Builds whichever of the two libraries and the marshalling module is missing or
    older than its sources (all with force); returns the path of the regular library."""
    todo = [(LIB, [], "release"), (LIB_DEBUG, ["-DMOE_DEBUG"], "debug")]
    todo = [v for v in todo if force or _stale(v[0])]
    if todo:
        _build_variants(todo, verbose, ptxas_verbose)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
