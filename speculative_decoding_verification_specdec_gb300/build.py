"""Build libspecdec.so in-tree with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("specdec_verify.cu", "specdec_ngram.cu", "specdec_bitmask.cu",
                                                  "specdec_rope.cu", "specdec_kvcache.cu", "specdec_attention.cu",
                                                  "specdec_top.cu", "specdec_distill.cu")]
HEADERS = [os.path.join(PKG, "csrc", f) for f in ("specdec_rows.cuh", "specdec_tensor.cuh", "specdec_logits.cuh")] + [os.path.join(ROOT, "include", "specdec.h")]
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libspecdec.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA 13 toolkit required)")


def _run(cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({' '.join(cmd)}):\n{res.stdout}\n{res.stderr}")
    return res.stdout + res.stderr


def build_library(out: str = LIB_PATH, extra_flags=(), verbose: bool = False) -> str:
    """Compile the sources side by side, then link them."""
    tmp = f"{out}.tmp{os.getpid()}"          # write then rename: concurrent builders never see a partial file
    with tempfile.TemporaryDirectory() as objects, concurrent.futures.ThreadPoolExecutor() as pool:
        objs = [os.path.join(objects, os.path.basename(s) + ".o") for s in SOURCES]
        compiled = pool.map(_run, ([nvcc(), *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-c", "-o", o, s]
                                   for s, o in zip(SOURCES, objs)))
        said = "".join(compiled) + _run([nvcc(), *NVCC_FLAGS, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    os.replace(tmp, out)
    if verbose:
        print(said)
    return out


def needs_rebuild(out: str = LIB_PATH) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = SOURCES + HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


if __name__ == "__main__":
    print(build_library(verbose=True))
