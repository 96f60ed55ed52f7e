"""The row planner's arithmetic at the ends of 32 bits, compiled for the CPU with traps on
signed overflow (tests/rows_edges_host.cpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SERVING = os.path.join(os.path.dirname(HERE), "decode_attention_09_b200", "csrc", "serving")


def test_planner_at_the_ends_of_32_bits(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = tmp_path / "rows_edges_host"
    subprocess.run([gxx, "-std=c++17", "-O1", "-ftrapv", "-I", SERVING,
                    os.path.join(HERE, "rows_edges_host.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"
