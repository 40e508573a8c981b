"""The short quotient's reciprocal over all scales that take it, on the host."""
import os
import shutil
import subprocess

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_reciprocal_is_as_near_as_it_says(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no g++ or no HIP headers")
    exe = str(tmp_path / "quotient")
    subprocess.run(["g++", "-std=gnu++17", "-O1", "-ffp-contract=off", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__", "-isystem",
                    "/opt/rocm/include", os.path.join(TESTS, "quotient_check.cpp"), "-o", exe], check=True)
    scales, worst, bad = map(int, subprocess.run([exe], text=True, capture_output=True, check=True).stdout.split())
    assert scales == 164 * 128       # 2^-64 up to 2^100
    assert bad == 0 and worst <= 2 ** 16     # 2^-44 in units of 2^-60
