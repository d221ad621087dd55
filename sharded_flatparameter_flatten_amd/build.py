"""Builds libfsdpshard.so in-tree with hipcc for gfx950.

The host indexer (csrc/unit.cpp) is plain C++; the kernels and their entry
points are HIP: csrc/kernels.hip (the shard step), csrc/muon_step.hip,
csrc/orthogonalize.hip, csrc/rms_norm.hip, csrc/embedding.hip, csrc/dropout.hip and
csrc/linear_cross_entropy.hip, compiled side by side. csrc/calls.cpp
becomes _calls.so, the extension module that marshals the shortest calls' tensors;
it links against the library beside it. Flags that fix the numerics:
-ffp-contract=off (no fused multiply-add anywhere on the path), the default
correctly rounded fp32 division and square root (never -ffast-math), and
packed-fp32 instructions disabled for device code.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libfsdpshard.so"
CALLS_NAME = "_calls.so"
SOURCES = ["unit.cpp", "kernels.hip", "muon_step.hip", "orthogonalize.hip", "rms_norm.hip", "embedding.hip",
           "dropout.hip", "linear_cross_entropy.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-Wall", "-I", INCLUDE, "-I", CSRC]
DEVICE = [f"--offload-arch={ARCH}", "-mcode-object-version=5",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
# The small products' first arguments arrive in registers (a launch 0.2 us shorter).
SOURCE_FLAGS = {"orthogonalize.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=8"]}


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"build step failed: {' '.join(cmd)}")
    noise = "is not a recognized feature for this target"
    rest = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if verbose and rest.strip():
        print(rest)


def build(out_dir: str | None = None, defines=(), verbose: bool = False) -> str:
    """Compiles the library; returns the path of the .so."""
    out_dir = out_dir or PKG
    obj_dir = os.path.join(out_dir, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    dflags = [f"-D{d}" for d in defines]

    def compile_one(source):
        obj = os.path.join(obj_dir, os.path.splitext(source)[0] + ".o")
        lang = ["-x", "hip", *DEVICE, *SOURCE_FLAGS.get(source, [])] if source.endswith(".hip") else ["-x", "c++"]
        _run([HIPCC, *lang, *COMMON, *dflags, "-c", os.path.join(CSRC, source), "-o", obj], verbose)
        return obj

    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    torch_include = os.path.join(torch_dir, "include")
    calls = os.path.join(obj_dir, "calls.o")
    includes = [sysconfig.get_paths()["include"], torch_include,
                os.path.join(torch_include, "torch", "csrc", "api", "include")]

    def compile_calls():
        _run([HIPCC, "-x", "c++", *COMMON, "-fvisibility=hidden", *[x for i in includes for x in ("-isystem", i)],
              "-c", os.path.join(CSRC, "calls.cpp"), "-o", calls], verbose)

    with ThreadPoolExecutor(8) as pool:
        binding = pool.submit(compile_calls)
        objects = list(pool.map(compile_one, SOURCES))
        binding.result()
    tmp = os.path.join(out_dir, LIB_NAME + ".tmp")
    _run([HIPCC, *DEVICE, "-shared", "-fPIC", "-o", tmp, *objects], verbose)
    final = os.path.join(out_dir, LIB_NAME)
    os.replace(tmp, final)
    tmp = os.path.join(out_dir, CALLS_NAME + ".tmp")
    _run([HIPCC, "-shared", "-fPIC", "-o", tmp, calls, "-L", out_dir, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"], verbose)
    os.replace(tmp, os.path.join(out_dir, CALLS_NAME))
    shutil.rmtree(obj_dir, ignore_errors=True)
    return final


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
