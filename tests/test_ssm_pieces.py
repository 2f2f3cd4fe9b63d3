"""The arithmetic by which the kernels of the causal convolution and the
selective scan find their rows from seq_start, and their places in them, built
from the kernels' own header by g++ with UndefinedBehaviorSanitizer and run
over valid and invalid values up to the largest problems that a plan accepts."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def test_rows_of_any_seq_start_stay_in_range_without_overflow(tmp_path):
    """A sequence that ends where T and L are 2^30 is the one whose end overflowed as a sum: its empty neighbour got 2^30
    rows past the end of every tensor."""
    exe = str(tmp_path / "pieces")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "sanitize", "ssm_pieces_driver.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
    assert int(r.stdout) > 100000
