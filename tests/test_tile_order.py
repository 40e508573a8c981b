"""Every tile is one workgroup's, whatever the size, in the order that
csrc/fp8tile_order.h gives the one-pass kernels."""
import tile_cases
from test_moe_paths import host_program


def test_every_tile_once(tmp_path):
    ask = host_program(tmp_path, "tile_order_dump.cpp")
    sizes = [(r, c) for r in (*range(1, 70), 113, 114, 127, 128, 129, 160, 256, 511, 512, 4096) for c in (*range(1, 34), 48, 64)]
    blocked = 0
    for (r, c), (b, groups, once, more) in zip(sizes, ask(sizes)):
        assert (once, more) == (r * c, 0), (r, c)
        # as many more find no tile as the rule allows; those beside a single narrow column of blocks do not count
        assert not b or groups * min(c, 8) <= 9 * r * c, (r, c)
        blocked += b
    assert 0 < blocked < len(sizes)


def test_sizes_of_the_gpu_tests(tmp_path):
    ask = host_program(tmp_path, "tile_order_dump.cpp")
    got = ask(tile_cases.BLOCKED)
    assert [g[0] for g in got] == [1] * len(got)
    assert {g[1] > r * c for (r, c), g in zip(tile_cases.BLOCKED, got)} == {True, False}
    assert [g[0] for g in ask([(tile_cases.PIECE, c) for _, c in tile_cases.BLOCKED])] == [0] * len(got)
