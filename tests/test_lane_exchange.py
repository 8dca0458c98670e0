"""Where lanes of a wavefront hand values to each other through LDS, the compiled products keep the
writes before the reads: the compiler, which sees one lane's addresses, is told so at each place. Looks at
the device code of the sources as the library compiles them (CPU only)."""
import os
import shutil
import subprocess

import pytest

from fp8_optimizer_state_amd import _build
from test_matrix_code import HIPCC


CODE = {}  # of a source, compiled once


def device_code(name, tmp_path):
    """Assembly of a source, its comments kept."""
    if name in CODE:
        return CODE[name]
    if shutil.which(HIPCC) is None:
        pytest.skip("needs hipcc")
    out = os.path.join(tmp_path, "device.s")
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    done = subprocess.run([HIPCC, *flags, "-I" + _build.INCLUDE, "--offload-device-only", "-S", "-o", out, os.path.join(_build.CSRC, name)],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    CODE[name] = open(out).read()
    return CODE[name]


def kernels(text, name):
    lines, at = text.splitlines(), None
    for i, line in enumerate(lines):
        if at is None and line.startswith("_Z") and name in line.split(":")[0] and ":" in line:
            at = i
        elif at is not None and line.startswith(".Lfunc_end"):
            yield lines[at].split(":")[0], [x.strip() for x in lines[at + 1:i]]
            at = None


def unordered(lines):
    """(reads of LDS behind a write with neither a barrier of the workgroup nor an ordering of the wavefront
    between them, such orderings behind a write)."""
    bad, orders, written = [], 0, False
    for line in lines:
        if line.startswith("; wave barrier"):
            orders += written
            written = False
        elif line.startswith("s_barrier"):
            written = False
        elif line.startswith("ds_write"):
            written = True
        elif line.startswith("ds_read") and written:
            bad.append(line)
    return bad, orders


def test_the_check_finds_what_is_missing():
    write, read, order = "ds_write_b128 v1, v[2:5]", "ds_read_b128 v[2:5], v1", "; wave barrier"
    assert unordered([write, order, read]) == ([], 1) and unordered([write, "s_barrier", read]) == ([], 0)
    assert unordered([read, write]) == ([], 0) and unordered([write, read])[0] == [read]


@pytest.mark.parametrize("name", ["linear.hip", "cross_entropy.hip"])
def test_tiles_leave_through_lds_in_order(name, tmp_path):
    seen = 0
    for kernel, lines in kernels(device_code(name, tmp_path), "product_tile_kernel"):
        bad, orders = unordered(lines)
        assert not bad, (kernel, bad[:3])
        if "LogSumOut" not in kernel:
            assert orders >= 1, kernel
            seen += 1
    assert seen >= 4


def test_the_4_bit_products_tiles_too(tmp_path):
    seen = 0
    for kernel, lines in kernels(device_code("mx4_matmul.hip", tmp_path), "mx4_matmul_tile_kernel"):
        bad, orders = unordered(lines)
        assert not bad and orders >= 2, (kernel, bad[:3])
        seen += 1
    assert seen >= 3
