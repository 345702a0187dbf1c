"""Build libfp4mi.so (all HIP sources for gfx950) in-tree.

Usage: python block_scaled_fp4_amd/build.py   (or call build()).
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp4mi.so")
SOURCES = ["quant.hip", "fp4quant.hip", "fp8col.hip", "matmul.hip", "wgrad.hip", "rmsnorm.hip",
           "fp8quant.hip", "fp8mat.hip", "swiglu.hip", "router.hip", "abi.hip"]

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-fno-gpu-flush-denormals-to-zero", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def build(verbose=False):
    """Every source to an object of its own, side by side, then one library."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as out, concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(out, s + ".o") for s in SOURCES]
        common = [hipcc(), *FLAGS]
        cmds = [[*common, "-c", "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objects)]
        done = list(pool.map(lambda c: _run(c, verbose), cmds))
        done.append(_run([*common, "-shared", *objects, "-o", tmp], verbose) if all(done) else False)
    if not all(done):
        raise RuntimeError("hipcc failed building libfp4mi.so")
    os.replace(tmp, LIB)
    return LIB


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
    return r.returncode == 0


if __name__ == "__main__":
    print(build(verbose=True))
