"""The 4-bit cache's entry points from plain C: tests/c_abi/kv4_check.c builds
against include/fa.h alone, links the library and gets the documented status
codes (no GPU involved)."""
import os
import shutil
import subprocess

import pytest

import io_aware_exact_21_b200 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_plain_c_caller(tmp_path):
    lib = fa.library_path()
    fa.load_library()
    exe = tmp_path / "kv4_check"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                           "-I", "/usr/local/cuda/include", os.path.join(ROOT, "tests", "c_abi", "kv4_check.c"),
                           "-o", str(exe), lib, "-Wl,-rpath," + os.path.dirname(lib)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"
