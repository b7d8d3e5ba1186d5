"""Build step, in-tree: the CUDA library (csrc/fp8bs_lib.cu -> libfp8bs.so, with
nvcc alone) and, where torch is installed, the extension module over it that
ops.py calls for the norm and the 4-bit operators (csrc/binding.cpp ->
_binding.<Python's ABI>.torch-<version>.so).  The module's name holds what it was
built for: after another torch or Python is installed it is built again.

The library is compiled for sm_100a only (B200), no fast-math: the
quantization's fp32 division and reciprocal must be IEEE round-to-nearest.
"""
import importlib
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "fp8bs_lib.cu")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libfp8bs.so")
BINDING = os.path.join(SRC_DIR, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def _sources():
    out = [os.path.join(INCLUDE, "fp8bs.h")]
    for f in sorted(os.listdir(SRC_DIR)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(SRC_DIR, f))
    return out


def _older(path: str, sources) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in sources)


def needs_build() -> bool:
    return _older(LIB_PATH, _sources())


def _run(cmd, path: str):
    """Runs cmd with a temporary output, which then takes path's place."""
    tmp = path + f".tmp{os.getpid()}"
    subprocess.run([*cmd, "-o", tmp], check=True)
    os.replace(tmp, path)


def binding_path() -> str:
    """The extension module for this Python and the installed torch."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = importlib.import_module("torch").__version__
    return os.path.join(HERE, f"_binding.{sysconfig.get_config_var('SOABI')}.torch-{version}.so")


def _build_binding(torch: str):
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
          "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"),
          "-isystem", os.path.join(cuda, "include"), BINDING, "-L", HERE, "-l:libfp8bs.so",
          "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
          "-Wl,-rpath,$ORIGIN"], binding_path())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or needs_build():
        cmd = [os.environ.get("NVCC", "nvcc"), *NVCC_FLAGS, "-I", INCLUDE, MAIN]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        _run(cmd, LIB_PATH)
    torch = importlib.util.find_spec("torch")
    if torch is not None and (force or _older(binding_path(), [BINDING, os.path.join(INCLUDE, "fp8bs.h")])):
        _build_binding(torch.submodule_search_locations[0])
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
