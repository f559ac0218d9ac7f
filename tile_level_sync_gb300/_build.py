"""In-tree build of the CUDA library (libcusync.so) for sm_103a with nvcc.

One -gencode; the translation units are compiled side by side and linked into a shared
object next to this file.  Rebuilds when any source or public header is newer than the
library.
"""

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")          # the chains
CSRC_MOE = os.path.join(PKG, "csrc_moe")  # the expert layer
INCLUDE = os.path.join(ROOT, "include")
OBJECTS = os.path.join(PKG, "build")
LIB_PATH = os.path.join(PKG, "libcusync.so")

SOURCES = [os.path.join(CSRC, "cusync.cu")] + [
    os.path.join(CSRC_MOE, f) for f in ("moe.cu", "moe_route_f32.cu", "moe_route_bf16.cu")]
DEPS = SOURCES + [
    os.path.join(d, f) for d in (CSRC, CSRC_MOE) for f in sorted(os.listdir(d)) if f.endswith((".h", ".cuh"))
] + [os.path.join(INCLUDE, f) for f in ("cusync.h", "cusync_moe.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I" + INCLUDE,
]


def _nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcusync.so")


def needs_build():
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in DEPS)


def build(force=False, verbose=False, extra_flags=()):
    """Compile libcusync.so if it is missing or stale; return its path."""
    if not force and not needs_build():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(OBJECTS, exist_ok=True)
    objs = [os.path.join(OBJECTS, os.path.splitext(os.path.basename(src))[0] + ".o") for src in SOURCES]
    running = []
    for src, obj in zip(SOURCES, objs):
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    outputs = [(p.communicate()[0], p.returncode) for p in running]
    tmp = LIB_PATH + ".tmp"
    if all(rc == 0 for _, rc in outputs):
        cmd = [nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        outputs.append((res.stdout + res.stderr, res.returncode))
    if any(rc != 0 for _, rc in outputs):
        raise RuntimeError("nvcc failed:\n" + "".join(text for text, _ in outputs))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
