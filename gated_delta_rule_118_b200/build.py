"""Build libgdn2.so (the C-ABI library) in-tree with nvcc for sm_100a, and the Python
module that calls it (_call.so) with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIBRARY = PKG / "libgdn2.so"
CALLER = PKG / "_call.so"
OBJDIR = PKG / "_build"

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-v", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = Path(os.environ.get("CUDA_HOME", "/usr/local/cuda")) / "bin" / "nvcc"
    return str(cand) if cand.exists() else "nvcc"


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _deps() -> list[Path]:
    return sources() + sorted(CSRC.glob("*.c")) + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + sorted(INCLUDE.glob("*.h"))


def is_stale() -> bool:
    if not LIBRARY.exists() or not CALLER.exists():
        return True
    t = min(LIBRARY.stat().st_mtime, CALLER.stat().st_mtime)
    return any(p.stat().st_mtime > t for p in _deps())


def build_library(force: bool = False, verbose: bool = False) -> Path:
    """Compile every csrc/*.cu to an object and link them into libgdn2.so; compile _call.so."""
    if not force and not is_stale():
        return LIBRARY
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
    caller = CALLER.with_suffix(".so.tmp")
    host = [os.environ.get("CC", "gcc"), "-O2", "-std=gnu11", "-shared", "-fPIC", "-Wall", "-Wno-unused-parameter",
            f"-I{sysconfig.get_paths()['include']}", f"-I{INCLUDE}", str(CSRC / "binding.c"), "-o", str(caller)]
    r = subprocess.run(host, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{host[0]} failed on binding.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    os.replace(caller, CALLER)
    (OBJDIR / "ptxas.log").write_text("\n".join(logs))
    if verbose:
        print("\n".join(logs))
    return LIBRARY


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIBRARY)
