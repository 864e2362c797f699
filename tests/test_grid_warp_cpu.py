"""The split merge's warp numbering, built for the host with g++
(tests/host/grid_warp_check.cc), and the sizes past it that are refused."""
import os
import shutil
import subprocess

import pytest

import io_aware_exact_21_b200 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_warps_are_numbered_past_2_27(tmp_path):
    exe = tmp_path / "grid_warp_check"
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror",
                           "-I", os.path.join(ROOT, "io_aware_exact_21_b200", "csrc"),
                           os.path.join(ROOT, "tests", "host", "grid_warp_check.cc"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"


def test_more_rows_and_heads_than_warps_are_refused():
    # 2^33 (query, head) pairs of d = 64
    assert fa.fa_fwd_kv4(P, P, P, P, P, P, P, 1, 8, 8, 1 << 30, 64, 64, 0.1, 1, 0, None, 2, None, 0, 0) == -3
    assert fa.fa_fwd_kv4_workspace_size(1, 8, 8, 1 << 30, 64, 64, 0, 2) == 0
