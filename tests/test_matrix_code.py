"""The compiled products: their matrix instructions are written out in the source, so that
the compiler adds no waits for them. Looks at the device code of the sources as the
library compiles them (CPU only)."""
import os
import re
import shutil
import subprocess

import pytest

from fp8_optimizer_state_amd import _build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def registers(operand: str):
    m = re.match(r"([av])\[(\d+):(\d+)\]$", operand)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"([av])(\d+)$", operand)
    return {(m.group(1), int(m.group(2)))} if m else set()


def kernels(text: str):
    for m in re.finditer(r"^(_Z\S*product_tile_kernel\S*):.*?^\.Lfunc_end", text, re.M | re.S):
        yield m.group(1), [line.split(";")[0].strip() for line in m.group(0).splitlines()[1:]]


def faults(lines):
    """Places where an operand was written by a vector instruction within the two states before, or where
    something other than a matrix instruction touches accumulators too soon after one."""
    bad, matrix = [], 0
    recent = []     # registers written by vector instructions, by states ago
    pending = {}    # accumulators of matrix instructions: states since
    for line in lines:
        if not line or line.endswith(":") or line.startswith(".") or line.startswith("#"):
            continue
        op, _, rest = line.partition(" ")
        operands = [o.strip().split(" ")[0] for o in rest.split(",")]
        states = int(operands[0]) + 1 if op == "s_nop" else 1
        if op.startswith("v_mfma_f32_16x16x32"):
            matrix += 1
            reads = set().union(*(registers(o) for o in operands[1:4]))
            if any(reads & w for w in recent[-2:]):
                bad.append(line)
        elif not op.startswith("s_") and op.split("_")[0] in ("v", "ds", "global", "scratch", "buffer", "flat"):
            touched = set().union(*(registers(o) for o in operands))
            if any(r in pending and pending[r] < 20 for r in touched):
                bad.append(line)
        written = registers(operands[0]) if op.startswith("v_") and not op.startswith("v_mfma") and not op.startswith("v_cmp") else set()
        recent.append(written)
        recent.extend([set()] * (states - 1))
        del recent[:-4]
        for r in list(pending):
            pending[r] += states
            if pending[r] > 40:
                del pending[r]
        if op.startswith("v_mfma_f32_16x16x32"):
            for r in registers(operands[0]):
                pending[r] = 0
    return bad, matrix


def test_the_check_finds_faults():
    good = ["ds_read_b128 v[0:3], v9", "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"]
    assert faults(good) == ([], 1)
    assert faults(["v_mov_b32_e32 v5, v20", "s_nop 0"] + good)[0] == []
    assert len(faults(good[:1] + ["v_mov_b32_e32 v5, v20"] + good[1:])[0]) == 1
    assert len(faults(["v_accvgpr_write_b32 a1, 0", "s_nop 0"] + good[1:])[0]) == 1
    assert faults(["v_accvgpr_write_b32 a1, 0", "s_nop 1"] + good[1:])[0] == []
    assert len(faults(good + ["v_accvgpr_read_b32 v1, a2"])[0]) == 1
    assert faults(good + ["s_nop 15", "s_nop 15", "v_accvgpr_read_b32 v1, a2"])[0] == []


@pytest.mark.parametrize("name", ["linear.hip", "cross_entropy.hip"])
def test_operands_and_results_of_matrix_instructions_settle(name, tmp_path):
    if shutil.which(HIPCC) is None:
        pytest.skip("needs hipcc")
    out = os.path.join(tmp_path, "device.s")
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    done = subprocess.run([HIPCC, *flags, "-I" + _build.INCLUDE, "--offload-device-only", "-S", "-o", out, os.path.join(_build.CSRC, name)],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    seen = 0
    for kernel, lines in kernels(open(out).read()):
        bad, matrix = faults(lines)
        assert matrix >= 32, kernel
        assert not bad, (kernel, bad[:5])
        seen += 1
    assert seen >= 4
