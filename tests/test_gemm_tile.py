"""The general GEMM's scale bytes in LDS: every lane's words lie on a multiple of
their size, inside the scales, and hold the lane's own rows."""
import os
import shutil
import subprocess

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_scale_bytes_are_read_where_they_are(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "tile")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", os.path.join(TESTS, "gemm_tile_check.cpp"),
                    "-o", exe], check=True)
    lines = [line.split() for line in subprocess.run([exe], text=True, capture_output=True, check=True).stdout.splitlines()]
    assert len(lines) == 8
    for name, off, past, other in lines:
        assert (off, past, other) == ("0", "0", "0"), name
