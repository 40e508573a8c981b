"""Which kernels the operators of include/fp8moe.h take at which sizes, from
the library's own rules compiled for the host."""
import os
import shutil
import subprocess

import numpy as np
import pytest

import moe_cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_fp8_linear_amd", "csrc")
POW2, FP32 = 0, 1


def host_program(tmp_path, source, *others):
    """Compile tests/<source> for the host; a function from input lines of numbers to output lines of numbers."""
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no g++ or no HIP headers")
    exe = str(tmp_path / "paths")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-isystem",
                    "/opt/rocm/include", os.path.join(ROOT, "tests", source), *(os.path.join(CSRC, o) for o in others),
                    "-o", exe], check=True)

    def ask(lines):
        r = subprocess.run([exe], input="".join(" ".join(map(str, line)) + "\n" for line in lines), text=True,
                           capture_output=True, check=True, timeout=60)
        got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(lines)
        return got
    return ask


def test_linear_takes_a_gemm_by_the_kernel_it_would_be(tmp_path):
    """The block-scaled GEMM from about 7.5 million outputs on; the general one,
    which is what amax / 448 scales and some reductions get, from 40 million,
    beyond a reduction of 6144 from 28 million (2 more each where rows beyond a
    multiple of 128 are left over)."""
    block = [(2048, 4096, 2048), (768, 12288, 512), (3000, 9216, 2048), (1920, 4096, 16384), (2560, 4096, 8192)]
    below = [(1536, 4096, 2048), (2000, 4096, 8192), (127, 65536, 512)]
    general = [(4096, 10240, 640), (8192, 5120, 4224), (4096, 12288, 16896), (3500, 12288, 640)]
    short = [(2048, 4096, 4224), (3000, 9216, 640), (4096, 7680, 4224), (3000, 9216, 16896), (3400, 12288, 640)]
    want = {(*s, POW2): s[0] // 128 * 128 for s in block + general}
    want.update({(*s, POW2): 0 for s in below + short})
    want.update({(*s, FP32): s[0] // 128 * 128 for s in general + [(4096, 10240, 2048), (4096, 7680, 8192), (2500, 12288, 6400)]})
    want.update({(*s, FP32): 0 for s in block + below + short})
    got = host_program(tmp_path, "linear_paths_check.cpp", "api_moe.cpp")(list(want))
    for (M, N, K, mode), (rc, gemm, rows) in zip(want, got):
        assert rc == 0 and gemm == want[M, N, K, mode] and gemm + rows == M, (M, N, K, mode, gemm, rows)


def test_every_kernel_is_reached(tmp_path):
    ask = host_program(tmp_path, "moe_plan_dump.cpp")
    gate, down = set(), set()
    for few, _, _, gt, _, gs, dt, _, ds in ask([(1, *s, mode) for s in moe_cases.WIDE for mode in (POW2, FP32)]):
        assert not few
        gate.add((gt, gs))
        down.add((dt, ds))
    assert gate == {(1, 2), (1, 4), (2, 2), (2, 3), (4, 2), (4, 3)}
    assert down == {(1, 2), (1, 3), (2, 2), (2, 4), (4, 2), (4, 4)}
    for shape, got in zip(moe_cases.NARROW, ask([(1, *s, POW2) for s in moe_cases.NARROW])):
        assert got[0] and got[1] < got[2], (shape, got)
    got = ask([(0, *s, POW2) for s in moe_cases.LINEAR_WIDE + moe_cases.LINEAR_TILES])
    assert not any(raw for raw, *_ in got)
    assert {tuple(tile) for _, *tile in got} == {
        (8, 8, 4, 4), (8, 8, 4, 2), (16, 1, 1, 0), (8, 2, 1, 0), (8, 2, 2, 0), (8, 4, 2, 0), (8, 4, 4, 0), (4, 3, 2, 0),
        (4, 4, 2, 0)}
    paths = host_program(tmp_path, "linear_paths_check.cpp", "api_moe.cpp")
    for (M, _, _), (rc, gemm, rows) in zip(moe_cases.LINEAR_GEMM, paths([(*s, POW2) for s in moe_cases.LINEAR_GEMM])):
        assert rc == 0 and gemm == M // 128 * 128 and rows == M % 128 > 0


@pytest.mark.parametrize("T,H,I,E,k", moe_cases.WIDE)
def test_uneven_ids(T, H, I, E, k):
    ids = moe_cases.uneven_ids(T, E, k, 1)
    assert all(len({e for e in row if e >= 0}) == (row >= 0).sum() for row in ids)
    counts = set(np.bincount(ids[ids >= 0], minlength=E).tolist())
    assert {0, 1, 15, 16, 17, 31, 32, 33} <= counts and (T < 80 or {47, 48, 49, 63, 64, 65, 80} <= counts)
