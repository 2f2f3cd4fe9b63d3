"""csrc/ssm.cpp (entry points of the causal convolution and the selective scan)
built by g++ with AddressSanitizer, with each of its host allocations failing
in turn: no exception crosses the C boundary, and the error has a reason."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "grouped_convolution_backward_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def test_a_failed_allocation_is_an_error_with_a_reason(tmp_path):
    exe = str(tmp_path / "memory")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                        os.path.join(CSRC, "ssm.cpp"), os.path.join(ROOT, "tests", "sanitize", "ssm_memory_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:detect_leaks=1:alloc_dealloc_mismatch=0")
    r = subprocess.run([exe], capture_output=True, text=True, env=env)
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
    assert int(r.stdout) >= 4
