"""The sizes of tests/expert_cases.py take the tiles that they are there for."""
import expert_cases
from test_moe_paths import FP32, POW2, host_program

WAYS = ("fprop", "dgrad", "wgrad")


def test_tiles(tmp_path):
    ask = host_program(tmp_path, "train_paths_dump.cpp", "plan.cpp")
    line = lambda way, N, K, E, R: (WAYS.index(way), R, N, K, E)  # noqa: E731
    got = [g[0] for g in ask([(*line(*size), POW2, 0) for size, _ in expert_cases.SIZES])]
    assert got == [tiles for _, tiles in expert_cases.SIZES]
    got = [g[0] for g in ask([(*line(*size), FP32, 0) for size, _ in expert_cases.SIZES])]
    assert got == [expert_cases.SMALL if tiles == expert_cases.LARGE else tiles for _, tiles in expert_cases.SIZES]


def test_spreads():
    for (_, _, _, E, R), _ in expert_cases.SIZES:
        e, lists = expert_cases.spreads(E, R)
        assert len({tuple(lengths) for lengths in lists}) == 4
        assert all(lengths[e] == expert_cases.MIDDLE and len(lengths) == E and sum(lengths) <= R for lengths in lists)


def test_spreads_with_tiles_of_256_rows_and_of_128():
    """A rows product on the large tiles takes tiles of 128 rows alone where there are at most 256 of them."""
    for (way, N, K, E, R), tiles in expert_cases.SIZES:
        if tiles == expert_cases.LARGE and way != "wgrad":
            columns = -(-(N if way == "fprop" else K) // 256)
            blocks = [sum(lengths) // 128 for lengths in expert_cases.spreads(E, R)[1]]
            assert {b * columns <= 256 for b in blocks} == {True, False}
