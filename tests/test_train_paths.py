"""Which kernels the operators of include/fp8train.h take at which sizes, from
the library's own rules compiled for the host."""
import train_cases
from test_moe_paths import FP32, POW2, host_program

LARGE, SMALL, FEW = range(3)
WAYS = ("fprop", "dgrad", "wgrad")


def test_every_kernel_of_the_grouped_products_is_reached(tmp_path):
    ask = host_program(tmp_path, "train_paths_dump.cpp", "plan.cpp")
    lines = [(WAYS.index(way), train_cases.rows(lengths, behind), N, K, len(lengths), mode, 0)
             for way, N, K, lengths, behind in train_cases.GROUPED for mode in (POW2, FP32)]
    got = ask(lines)
    reached = {(WAYS[line[0]], line[5], g[0]) for line, g in zip(lines, got)}
    want = {(way, mode, tiles) for way in ("fprop", "dgrad") for mode in (POW2, FP32) for tiles in (SMALL, FEW)}
    want |= {("fprop", POW2, LARGE), ("dgrad", POW2, LARGE), ("wgrad", POW2, LARGE), ("wgrad", POW2, SMALL),
             ("wgrad", FP32, SMALL)}
    assert reached == want
    large = {(line[4] > 256, g[1] > 1) for line, g in zip(lines, got) if line[0] == 2 and g[0] == LARGE}
    assert {(False, True), (True, True), (False, False)} <= large


def test_wgrads_rules(tmp_path):
    """What its comments measured, and what the large tiles cannot take."""
    ask = host_program(tmp_path, "train_paths_dump.cpp", "plan.cpp")
    large = [(73728, 2048, 2048, 64), (10240, 2048, 2048, 64), (6144, 4096, 1024, 16), (81920, 768, 2048, 128)]
    small = [(1792, 1280, 1152, 11), (7168, 896, 3328, 52), (39936, 1408, 256, 44), (512, 512, 512, 8)]
    off = [(73728 + 128, 2048, 2048, 64), ((1 << 22) + 512, 2048, 2048, 64)]
    assert [g[0] for g in ask([(2, *s, POW2, 0) for s in large])] == [LARGE] * 4
    assert [g[0] for g in ask([(2, *s, POW2, 0) for s in small + off])] == [SMALL] * 6
    assert [g[0] for g in ask([(2, *s, POW2, 1) for s in large])] == [SMALL] * 4
    assert [g[0] for g in ask([(2, *s, FP32, 0) for s in large])] == [SMALL] * 4


def test_gather_in_the_order_of_tokens(tmp_path):
    ask = host_program(tmp_path, "train_paths_dump.cpp", "plan.cpp")
    yes = [(16384, 2048, 147456, 8, 0), (4000, 1408, 66560, 16, 0), (65536, 4224, 1 << 20, 16, 0)]
    no = [(2048, 2048, 24576, 8, 0),        # x fits two XCDs' L2
          (16384, 2048, 147456, 8, 1),      # both orientations
          (16384, 2048, 24576, 1, 0),       # each row once
          (8192, 2048, 36864, 4, 0),        # too little read again
          (16384, 2048, 1 << 22, 8, 0)]     # runs longer than a wave
    assert [g[0] for g in ask([(3, *s) for s in yes])] == [1] * 3
    assert [g[0] for g in ask([(3, *s) for s in no])] == [0] * 5
