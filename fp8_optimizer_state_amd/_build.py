"""Build step for the HIP library (hipcc, gfx950)."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
# the step kernels, state codec and core ABI; the activation codec; the 4-bit
# codec and its product; the norms at a block's border
SOURCES = [os.path.join(CSRC, name) for name in
           ("coat_fp8.hip", "act_fp8.hip", "mx4.hip", "mx4_matmul.hip", "block_norm.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcoat_fp8.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # explicit fma only: the fp64 moment chain must not be re-associated
    "-ffp-contract=off",
    # no packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def build(verbose: bool = False) -> str:
    """Compile the csrc/*.hip sources into libcoat_fp8.so next to this file."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(src) + ".o") for src in SOURCES]

        def run(cmd):
            return subprocess.run(cmd, capture_output=True, text=True)

        # one compiler per source at a time, then one link
        compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
        with ThreadPoolExecutor(max_workers=4) as pool:
            done = list(pool.map(run, ([hipcc, *compile_flags, "-I" + INCLUDE, "-c", "-o", o, src]
                                       for src, o in zip(SOURCES, objects))))
        if all(res.returncode == 0 for res in done):
            done.append(run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *objects]))
    for res in done:
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print("".join(res.stderr for res in done))
    os.replace(tmp, LIB)
    return LIB


def build_ceiling_probe() -> str:
    """Compile bench_ceiling.hip (the memory-pattern instrument of bench.py
    --ceiling, not part of the library) into libbench_ceiling.so at the root."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    out = os.path.join(ROOT, "libbench_ceiling.so")
    flags = [f for f in HIPCC_FLAGS if f != "-ffp-contract=off"]
    res = subprocess.run([hipcc, *flags, "-o", out + ".tmp", os.path.join(ROOT, "bench_ceiling.hip")],
                         capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
