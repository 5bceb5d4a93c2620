"""Build libdg.so (the sm_100a CUDA library behind include/dg.h) in-tree with nvcc, and
_dgcall.so (argument marshalling of the binding's frequent calls) with g++, where g++ and torch's
C++ headers are at hand: libdg.so and the calls that start from m_indices or masked_m work without it."""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdg.so")
SOURCES = [os.path.join(CSRC, "dg_api.cu")]
CALL_LIB = os.path.join(HERE, "_dgcall.so")
CALL_SOURCE = os.path.join(CSRC, "dg_pycall.cpp")
HEADER = os.path.join(ROOT, "include", "dg.h")
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")] + [HEADER]


def nvcc_path() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def command(out: str = LIB, verbose_ptxas: bool = False) -> list:
    cmd = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-I", os.path.join(ROOT, "include"), "-o", out] + SOURCES
    if verbose_ptxas or os.environ.get("DG_PTXAS_VERBOSE") == "1":
        cmd[1:1] = ["-Xptxas", "-v"]
    return cmd


def call_command(out: str = CALL_LIB) -> list:
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [a for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
           for a in ("-isystem" if d != os.path.join(ROOT, "include") else "-I", d)]
    return ["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, CALL_SOURCE, "-o", out,
            "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", f"-Wl,-rpath,{lib}"]


def call_unavailable() -> str:
    """Why the extension cannot be built here ("": it can)."""
    if not shutil.which("g++"):
        return "no g++"
    try:
        from torch.utils import cpp_extension
    except ImportError:
        return "no torch"
    header = os.path.join("torch", "csrc", "autograd", "python_variable.h")
    if not any(os.path.exists(os.path.join(d, header)) for d in cpp_extension.include_paths()):
        return "no C++ headers of torch"
    return ""


def call_tag() -> str:
    """What the extension's binary interface depends on, kept beside it: the Python and the torch it is built for."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return f"{sysconfig.get_config_var('SOABI')} torch {torch}\n"


def call_up_to_date() -> bool:
    if not _newer(CALL_LIB, [CALL_SOURCE, HEADER]):
        return False
    try:
        with open(CALL_LIB + ".tag") as f:
            return f.read() == call_tag()
    except OSError:
        return False


def _newer(out: str, deps: list) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps if os.path.exists(d))


def up_to_date() -> bool:
    return _newer(LIB, DEPS)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or not up_to_date():
        subprocess.run(command(verbose_ptxas=verbose_ptxas), check=True)
    if force or not call_up_to_date():
        why = call_unavailable()
        if why:
            print(f"{CALL_LIB} is not built ({why}): routing, dispatch, combine and checkpoint calls need it",
                  file=sys.stderr)
        else:
            subprocess.run(call_command(CALL_LIB), check=True)
            with open(CALL_LIB + ".tag", "w") as f:
                f.write(call_tag())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
