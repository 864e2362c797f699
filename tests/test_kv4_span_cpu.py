"""The 4-bit cache's tile and mask arithmetic, built for the host with g++
(tests/host/kv4_span_check.cc): against 64-bit arithmetic at lengths and windows
up to 2^31 - 1, with signed overflow trapped."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_tiles_and_masks_up_to_the_last_row(tmp_path):
    exe = tmp_path / "kv4_span_check"
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow",
                           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "io_aware_exact_21_b200", "csrc"),
                           os.path.join(ROOT, "tests", "host", "kv4_span_check.cc"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"
