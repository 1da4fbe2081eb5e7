"""Build libgdn2.so (the C-ABI library) in-tree with nvcc for sm_100a, and with the host
compiler the Python module that calls it with less overhead than ctypes (_call, one
file an interpreter; the library serves without it)."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIBRARY = PKG / "libgdn2.so"
CALLER = PKG / f"_call{sysconfig.get_config_var('EXT_SUFFIX')}"  # (the interpreter's own: its version is in the name)
OBJDIR = PKG / "_build"

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-v", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = Path(os.environ.get("CUDA_HOME", "/usr/local/cuda")) / "bin" / "nvcc"
    return str(cand) if cand.exists() else "nvcc"


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _older(built: Path, deps: list[Path]) -> bool:
    return not built.exists() or any(p.stat().st_mtime > built.stat().st_mtime for p in deps)


def is_stale() -> bool:
    """Whether libgdn2.so is missing or older than its sources."""
    return _older(LIBRARY, sources() + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + sorted(INCLUDE.glob("*.h")))


def build_caller(force: bool = False) -> Path:
    """Compile csrc/binding.c for this interpreter; raises RuntimeError where that cannot be done."""
    if not force and not _older(CALLER, [CSRC / "binding.c", *INCLUDE.glob("*.h")]):
        return CALLER
    tmp = CALLER.with_suffix(".tmp")
    host = [os.environ.get("CC", "gcc"), "-O2", "-std=gnu11", "-shared", "-fPIC", "-Wall", "-Wno-unused-parameter",
            f"-I{sysconfig.get_paths()['include']}", f"-I{INCLUDE}", str(CSRC / "binding.c"), "-o", str(tmp)]
    try:
        r = subprocess.run(host, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{host[0]} cannot be run: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{host[0]} failed on binding.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLER)
    return CALLER


def build_library(force: bool = False, verbose: bool = False) -> Path:
    """Compile every csrc/*.cu to an object and link them into libgdn2.so; then compile the calling
    module, without which (no host compiler, no headers of Python) the library is as good, only its
    calls from Python take some microseconds longer."""
    if force or is_stale():
        _build_library(verbose)
    try:
        build_caller(force)
    except RuntimeError as e:
        warnings.warn(f"the hybrid block's operators are called through ctypes: {e}")
    return LIBRARY


def _build_library(verbose: bool) -> None:
    OBJDIR.mkdir(exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = OBJDIR / (src.stem + ".o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", str(src), "-o", str(obj)]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
        objs.append(obj)
    logs = []
    for src, p in procs:
        out, _ = p.communicate()
        logs.append(f"== {src.name}\n{out}")
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{out}")
    tmp = LIBRARY.with_suffix(".so.tmp")
    link = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *map(str, objs), "-o", str(tmp)]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    (OBJDIR / "ptxas.log").write_text("\n".join(logs))
    if verbose:
        print("\n".join(logs))


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIBRARY)
