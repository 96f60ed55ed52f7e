"""Build libgdattn.so in-tree: nvcc for sm_100a, static CUDA runtime, C ABI only."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgdattn.so")
SERVING = os.path.join(CSRC, "serving")
SOURCES = [os.path.join(CSRC, "api.cu"), os.path.join(SERVING, "serving.cu")]
OBJECTS = os.path.join(HERE, "_build")


def _headers(folder):
    return [os.path.join(folder, f) for f in sorted(os.listdir(folder))
            if f.endswith((".cuh", ".h"))]


# What each source is built from.
DEPS = {
    SOURCES[0]: [SOURCES[0], *_headers(CSRC), os.path.join(INCLUDE, "gdattn.h")],
    SOURCES[1]: [SOURCES[1], *_headers(CSRC), *_headers(SERVING),
                 os.path.join(INCLUDE, "gdattn.h")],
}

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
    "-Xcompiler", "-fPIC", "-cudart", "static", "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _older(path: str, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps)


def stale() -> bool:
    return any(_older(LIB, deps) for deps in DEPS.values())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile what changed (the sources side by side) and link the library."""
    if not force and not stale():
        return LIB
    os.makedirs(OBJECTS, exist_ok=True)
    objects, running = [], []
    for src, deps in DEPS.items():
        obj = os.path.join(OBJECTS, os.path.basename(src) + ".o")
        objects.append(obj)
        if not force and not _older(obj, deps):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", tmp]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        running.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = [cmd for proc, cmd, _, _ in running if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, tmp, obj in running:
        os.replace(tmp, obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", *objects, "-o", tmp], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
