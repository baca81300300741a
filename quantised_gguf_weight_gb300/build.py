"""Build the CUDA library libqk.so in-tree (nvcc, sm_103a only).

Each translation unit under csrc/ is compiled in parallel with
`-gencode arch=compute_103a,code=sm_103a`, then linked into
quantised_gguf_weight_gb300/_build/libqk.so against the CUDA runtime.
The calls from PyTorch tensors (csrc/qk_torch.cpp) are a CPython extension,
_build/qk_torch.so, compiled by g++ beside them against the headers of the
installed torch and linked to libqk.so; without torch there is only libqk.so.
Rebuilds only what a source or header is newer than, and the extension where it
was made for another torch or Python.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD_DIR, "libqk.so")
BINDING = os.path.join(BUILD_DIR, "qk_torch.so")
BINDING_FOR = os.path.join(BUILD_DIR, "qk_torch.for")      # the torch and Python that BINDING was made for
BINDING_SOURCE = os.path.join(CSRC, "qk_torch.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _newer_than(made: str, deps: list[str]) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(d) <= os.path.getmtime(made) for d in deps)


def _library_up_to_date() -> bool:
    return _newer_than(LIB, _deps())


def _torch_and_python() -> str:
    import torch
    return f"{torch.__version__} {os.path.dirname(torch.__file__)} {sys.implementation.cache_tag}"


def _binding_up_to_date() -> bool:
    try:
        with open(BINDING_FOR) as f:
            made_for = f.read()
    except OSError:
        return False
    return made_for == _torch_and_python() and \
        _newer_than(BINDING, [BINDING_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h")), os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _library_up_to_date() and (not _have_torch() or _binding_up_to_date())


def _binding_command(out: str) -> list[str]:
    """Compiles the extension to an object file: Python's and torch's own headers, nothing generated."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SOURCE, "-o", out,
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include")]


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    subprocess.check_call(["g++", "-shared", "-o", tmp, obj, "-L", BUILD_DIR, "-l:libqk.so", "-Wl,-rpath,$ORIGIN",
                           "-L", libs, f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
                           "-lc10_cuda"])
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_torch_and_python())


def _run(procs, verbose: bool) -> None:
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")


def build(force: bool = False, verbose: bool = False) -> str:
    library = force or not _library_up_to_date()
    binding = _have_torch() and (force or not _binding_up_to_date())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs, objs = [], []
    binding_obj = os.path.join(BUILD_DIR, "qk_torch.cpp.o")
    if binding:
        procs.append((BINDING_SOURCE, subprocess.Popen(_binding_command(binding_obj), stdout=subprocess.PIPE,
                                                       stderr=subprocess.STDOUT)))
    if library:
        nvcc = _nvcc()
        flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                        "--expt-relaxed-constexpr"]
        for src in sources():
            obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
            objs.append(obj)
            cmd = [nvcc, *flags, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    _run(procs, verbose)
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
    if binding:
        _link_binding(binding_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
