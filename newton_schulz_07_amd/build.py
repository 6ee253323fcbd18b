"""Compile libns_hip.so (gfx950) in-tree with hipcc.

    python -m newton_schulz_07_amd.build

The library is always rebuilt from source when this runs.
"""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libns_hip.so")

HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # multiply-adds fuse only where the source writes them as one expression
    # or fmaf, never by the backend's choice, so every kernel instance of the
    # same arithmetic rounds the same way
    "-ffp-contract=on",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]
SOURCES = ["ns_kernels.hip", "ns_peak.hip", "ns_noalloc.hip", "ns_norm.hip", "ns_route.hip", "ns_experts.hip",
           "ns_rms.hip", "ns_quantize.hip", "ns_experts_scaled.hip", "ns_host.cpp", "ns_api.cpp", "ns_sublayer.cpp",
           "ns_scaled.cpp"]


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def compile_source(src, tmp, verbose=False):
    obj = os.path.join(tmp, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [hipcc()] + HIP_FLAGS + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError(f"hipcc failed on {src}")
    if verbose:
        sys.stdout.write(r.stdout)
    return obj


def build(verbose=False):
    tmp = os.path.join(PKG, "_build")
    os.makedirs(tmp, exist_ok=True)
    with ThreadPoolExecutor(6) as pool:
        objs = list(pool.map(lambda src: compile_source(src, tmp, verbose), SOURCES))
    out_tmp = LIB + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", out_tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(out_tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
