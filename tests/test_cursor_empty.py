"""The walk over the offsets of packed sequences across many empty ones, on the
CPU."""
import os
import shutil
import subprocess

import pytest


def test_cursor_crosses_empty_sequences_in_few_reads(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    src = os.path.join(os.path.dirname(__file__), "csrc", "cursor_empty_check.cpp")
    exe = str(tmp_path / "cursor_empty_check")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
    assert r.returncode == 0, r.stdout + r.stderr
