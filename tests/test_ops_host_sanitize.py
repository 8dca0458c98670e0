"""The host-side logic of the layer-input operators (csrc/ops_host.h: argument checks, how
the border's backward pass deals rows to workgroups and the product its k) under
AddressSanitizer and UndefinedBehaviorSanitizer on the CPU. The library compiles the same
header."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_host_logic_clean_under_asan_ubsan(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = os.path.join(tmp_path, "ops_driver")
    built = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wno-unused-function", "-fno-omit-frame-pointer",
                            "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I" + os.path.join(ROOT, "include"),
                            "-I" + os.path.join(ROOT, "fp8_optimizer_state_amd", "csrc"), "-o", exe,
                            os.path.join(HERE, "sanitize", "ops_driver.cc")], capture_output=True, text=True)
    if built.returncode != 0 and "asan" in (built.stderr or "").lower():
        pytest.skip("the sanitizer runtime is not installed: " + built.stderr[-200:])
    assert built.returncode == 0, built.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    run = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert run.returncode == 0, (run.stdout + run.stderr)[-3000:]
    assert run.stdout.strip().endswith("ok")
