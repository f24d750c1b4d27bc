"""Build the sm_103a library liblk.so in-tree with nvcc (no torch extension
machinery): each .cu under csrc/ is compiled in parallel, then linked as one
shared library beside this file."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblk.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


# The files that make each kernel family (a stored profile of one stays valid
# while these are unchanged).
KERNEL_FILES = {
    "ring": ["lk_ring_kernel.cuh", "lk_ring.cu", "lk_ring_q0.cu", "lk_ring_q1.cu", "lk_ring_q2.cu"],
    "mma": ["lk_mma.cu", "lk_ring_kernel.cuh"],
    "chain": ["lk_chain.cu", "lk_ring_kernel.cuh"],
}
COMMON_FILES = ["lk_device.cuh", "lk_host.h"]


def sources_digest(kind: str | None = None) -> str:
    """sha256 over the sources and headers of one kernel family (or of the
    whole library): identifies the kernels a stored profile was taken on."""
    import hashlib
    h = hashlib.sha256()
    if kind is None:
        files = _sources() + _headers()
    else:
        files = [os.path.join(CSRC, f) for f in KERNEL_FILES[kind] + COMMON_FILES] + \
            [os.path.join(INCLUDE, "lk.h")]
    for p in files:
        with open(p, "rb") as f:
            h.update(os.path.basename(p).encode() + b"\0" + f.read())
    return h.hexdigest()


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


# Kernels that move registers between their warps at run time: the split is made
# for one number of registers at launch, which is the compiler's to choose (the
# library refuses to launch them with another).
SPLIT_KERNELS = {"lk_tile.cu": ("attn_tile_kernel", "kTileRegs")}


def check_registers(name, source, ptxas):
    """Raise if ptxas (its -v output) gave a kernel of SPLIT_KERNELS[name] another
    number of registers than the source's split is made for."""
    kernel, const = SPLIT_KERNELS[name]
    want = int(re.search(rf"\b{const} = (\d+)", source).group(1))
    got = re.findall(rf"entry function '([^']*{kernel}[^']*)'.*?Used (\d+) registers", ptxas, re.S)
    if not got:
        raise RuntimeError(f"{name}: no register counts of {kernel} in the output of ptxas")
    for fn, n in got:
        if int(n) != want:
            raise RuntimeError(f"{name}: {fn} has {n} registers at launch, its split is made for {want} ({const}): "
                               "with this compiler the split has to be made anew")


def _compile(src, verbose_ptxas):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if not _stale(obj, [src] + _headers() + [__file__]):
        return obj, ""
    split = os.path.basename(src) in SPLIT_KERNELS
    cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose_ptxas or split else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if split:
        try:
            with open(src) as f:
                check_registers(os.path.basename(src), f.read(), r.stderr)
        except RuntimeError:
            os.remove(obj)
            raise
    return obj, r.stderr


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    log = "".join(e for _, e in results)
    if log:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write(log)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
