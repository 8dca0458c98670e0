"""Operands that a call may be given as its output too are not promised to the compiler to lie apart
(CPU only: looks at the code that the sources compile to)."""
import os
import re
import shutil
import subprocess

import pytest

from fp8_optimizer_state_amd import _build
from test_matrix_code import HIPCC


def test_dropout_in_place(tmp_path):
    """y may be x or residual."""
    if shutil.which(HIPCC) is None:
        pytest.skip("needs hipcc")
    out = os.path.join(tmp_path, "device.ll")
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    done = subprocess.run([HIPCC, *flags, "-I" + _build.INCLUDE, "--offload-device-only", "-emit-llvm", "-S", "-o", out,
                           os.path.join(_build.CSRC, "dropout.hip")], capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    kernels = [line for line in open(out) if re.match(r"define .*amdgpu_kernel .*dropout_kernel", line)]
    assert len(kernels) == 8
    for line in kernels:
        assert "noalias" not in line, line[:200]
