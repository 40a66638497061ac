"""The tree attention's host tables are refused, with the reason, where their
lists or the work of making them pass a limit."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "prefix_tree_packed_plan_amd", "csrc")


def test_refusals_name_the_limit_that_was_passed(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "attn_plan_limits")
    cmd = [gxx, "-std=c++17", "-O1", os.path.join(ROOT, "tests", "attn_plan_limits.cpp"),
           os.path.join(CSRC, "attn_plan.cpp"), os.path.join(CSRC, "plan.cpp"), "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "limits hold" in run.stdout
