"""Build the C-ABI CUDA library ``libdap.so`` in-tree for sm_103a with nvcc, and the Python
extension ``_dap_torch.so`` (argument marshalling, csrc/dap_torch.cpp) with the host compiler.

Each translation unit is compiled in parallel, then linked.  The results land next to this
file; objects go to ``_build/``.  Rebuilds only when a source or header is newer than the
library, and the extension also when torch or Python are not those it was built for.  The
library needs nvcc only; the extension needs torch's headers and a built library.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdap.so")
EXT_SRC = os.path.join(CSRC, "dap_torch.cpp")
EXT = os.path.join(PKG, "_dap_torch.so")
EXT_FOR = os.path.join(BUILD, "_dap_torch.for")   # the torch and Python that EXT was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-O2", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer_than(path: str, inputs: list[str]) -> bool:
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    return os.path.exists(LIB) and _newer_than(LIB, _inputs())


def _ext_for() -> str:
    import torch

    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, Python {sys.version}"


def ext_fits() -> bool:
    """Whether the extension that is there was built for the torch and Python that run."""
    if not (os.path.exists(EXT) and os.path.exists(EXT_FOR)):
        return False
    with open(EXT_FOR) as f:
        return f.read() == _ext_for()


def ext_up_to_date() -> bool:
    return ext_fits() and _newer_than(EXT, [EXT_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _ext_flags() -> tuple[list[str], list[str]]:
    """Compile and link flags of the extension: torch's own headers and libraries."""
    import torch

    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda", "include"),
           INCLUDE]
    comp = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for d in inc:
        comp += ["-isystem" if d != INCLUDE else "-I", d]
    lib = os.path.join(root, "lib")
    link = [f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-L{PKG}", "-l:libdap.so",
            f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]
    return comp, link


def _run(cmd: list[str], what: str, verbose: bool = False) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """The library."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        _run([nvcc, *flags, "-c", src, "-o", obj], f"nvcc failed for {src}", verbose)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64",
          *objs, "-o", tmp], "link failed")
    os.replace(tmp, LIB)
    return LIB


def _compile_ext(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, os.path.basename(EXT_SRC) + ".o")
    cxx = os.environ.get("CXX", "g++")
    _run([cxx, *_ext_flags()[0], "-c", EXT_SRC, "-o", obj], f"{cxx} failed for {EXT_SRC}", verbose)
    return obj


def _link_ext(obj: str) -> str:
    tmp = EXT + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, *_ext_flags()[1]], "link failed")
    os.replace(tmp, EXT)
    with open(EXT_FOR, "w") as f:
        f.write(_ext_for())
    return EXT


def build_ext(force: bool = False, verbose: bool = False) -> str:
    """The extension, against the library that is there."""
    return EXT if not force and ext_up_to_date() else _link_ext(_compile_ext(verbose))


def build_all(force: bool = False, verbose: bool = False) -> None:
    """Both, compiled side by side."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        obj = None if not force and ext_up_to_date() else ex.submit(_compile_ext, verbose)
        build(force, verbose)
        if obj is not None:
            _link_ext(obj.result())


if __name__ == "__main__":
    build_all(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
