"""The way of a team of the tree kernel through a unit's items, run by threads of the CPU: waits that
run out for some of the threads let all of them leave at the same place."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_waits_that_run_out_leave_no_thread_at_a_barrier(tmp_path):
    exe = str(tmp_path / "tree_unit_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", os.path.join(HERE, "tree_unit_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
