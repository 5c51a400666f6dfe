"""Build libkronq.so in-tree with nvcc for sm_100a (B200), and _kv4.so, the torch
binding of its 4-bit cache calls, with the host compiler.

Usage: python -m post_quantization_02_b200.build [--force]
"""

from __future__ import annotations

import os
import pathlib
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = pathlib.Path(__file__).resolve().parent
SRC = HERE / "csrc"
INCLUDE = HERE.parent / "include"
OBJ = HERE / "_build"
LIB = HERE / "libkronq.so"
BINDING = HERE / "_kv4.so"
BINDING_SRC = SRC / "kv4_torch.cpp"

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-warn-spills",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkronq")


def _sources():
    return sorted(SRC.glob("*.cu"))


def _deps():
    return list(SRC.glob("*.cu")) + list(SRC.glob("*.cuh")) + list(INCLUDE.glob("*.h"))


def up_to_date() -> bool:
    if not LIB.exists():
        return False
    t = LIB.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in _deps())


def _build_binding(force: bool = False) -> None:
    """_kv4.so beside libkronq.so, which it finds by its own place."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    # the torch and the interpreter it is built against: another one's would not fit it
    against = f"{torch.__version__} {sys.version}"
    stamp = OBJ / "_kv4.built_against"
    if (not force and BINDING.exists() and BINDING.stat().st_mtime >= max(
            p.stat().st_mtime for p in (BINDING_SRC, *INCLUDE.glob("*.h")))
            and stamp.exists() and stamp.read_text() == against):
        return
    lib = pathlib.Path(torch.__file__).resolve().parent / "lib"
    cuda = pathlib.Path(nvcc()).resolve().parents[1]
    inc = [f"-I{p}" for p in (*cpp_extension.include_paths(), sysconfig.get_path("include"), cuda / "include")]
    tmp = BINDING.with_suffix(".so.tmp")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *inc, str(BINDING_SRC), "-o", str(tmp), f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           f"-L{HERE}", "-l:libkronq.so", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the torch binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    OBJ.mkdir(exist_ok=True)
    stamp.write_text(against)


def build(force: bool = False, verbose: bool = False) -> pathlib.Path:
    lib = _build_lib(force, verbose)
    _build_binding(force)
    return lib


def _build_lib(force: bool, verbose: bool) -> pathlib.Path:
    if not force and up_to_date():
        return LIB
    OBJ.mkdir(exist_ok=True)
    cc = nvcc()

    def compile_one(src: pathlib.Path):
        obj = OBJ / (src.stem + ".o")
        cmd = [cc, *NVCC_FLAGS, "-I", str(INCLUDE), "-c", str(src), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB.with_suffix(".so.tmp")
    cmd = [cc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", str(tmp),
           *map(str, objs), "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
