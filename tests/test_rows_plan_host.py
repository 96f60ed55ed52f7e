"""The row planner of the continuous-batching attention calls, run on the CPU.

csrc/serving/rows_plan.cuh and rows_chunks.cuh are copied beside an empty ptx.cuh
and compiled with g++ together with tests/rows_plan_host.cpp, which emulates the
warp intrinsics they use and checks, on random ragged batches, that every visible
position is in exactly one tile and slot, that chunks and segments cover every
tile once, and that the merges find exactly the pieces that were left.  A planted
mistake in a copy must make the check fail.
"""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SERVING = os.path.join(os.path.dirname(HERE), "decode_attention_09_b200", "csrc", "serving")
HEADERS = ("rows_plan.cuh", "rows_chunks.cuh")


def run_harness(tmp_path, cases, original=None, planted=None):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    found = 0
    (tmp_path / "serving").mkdir()
    (tmp_path / "ptx.cuh").write_text("// the planner uses none of the PTX wrappers\n")
    for name in HEADERS:
        with open(os.path.join(SERVING, name)) as f:
            text = f.read()
        if original is not None:
            found += text.count(original)
            text = text.replace(original, planted)
        (tmp_path / "serving" / name).write_text(text)
    assert original is None or found == 1
    exe = tmp_path / "rows_plan_host"
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wno-unknown-pragmas", "-I",
                    str(tmp_path / "serving"), "-I", HERE,
                    os.path.join(HERE, "rows_plan_host.cpp"), "-o", str(exe)], check=True)
    return subprocess.run([str(exe), str(cases)], capture_output=True, text=True, timeout=300)


def test_row_planner(tmp_path):
    r = run_harness(tmp_path, 400)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok 400"


@pytest.mark.parametrize("original,planted", [
    ("u.pin = imin32(g.sinks, lo);", "u.pin = g.sinks;"),
    ("u.run0 = imin32(hi - lo, g.capacity - u.slot0);", "u.run0 = hi - lo;"),
    ("UnitTiles u = {0, 0, 0, 0, 0, g.sinks, 0, 0, 1};",
     "UnitTiles u = {0, 0, 0, 0, 0, 0, 0, 0, 1};"),
    ("r.lo = g.window > 0 ? imax32(0, p + 1 - g.window) : 0;",
     "r.lo = g.window > 0 ? imax32(0, p - g.window) : 0;"),
    ("static_cast<int64_t>(P) + least_own + 1 - g.window",
     "static_cast<int64_t>(P) + least_own + 2 - g.window"),
    ("if (imax32(lo, g.sinks) < oldest) {", "if (lo < oldest - 2 * g.capacity - 100000) {"),
    ("return prefix_call ? c + unit : 2 * c + (opens ? 0 : 1);",
     "return prefix_call ? c + unit : 2 * c;"),
    ("if (first < begin) return false; ", "if (first < 0) return false; "),
    ("s.first = partial_slot(false, c, 0, start <= begin);",
     "s.first = partial_slot(false, c, 0, first <= begin);"),
    ("return static_cast<int32_t>(((static_cast<int64_t>(step) + 1) * n - 1) / steps);",
     "return static_cast<int32_t>(static_cast<int64_t>(step) * n / steps);"),
    ("s.opens = s.start <= plan->cs;", "s.opens = s.start < plan->cs;"),
    ("if (y_start + span > pos) break;", "if (y_start + span >= pos) break;"),
])
def test_planted_mistake_is_caught(tmp_path, original, planted):
    r = run_harness(tmp_path, 150, original, planted)
    assert r.returncode != 0, "the planted mistake went unnoticed"
