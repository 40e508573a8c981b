"""Sizes of experts' products by the tiles that they take (tests/test_expert_cases.py
checks that they do): (way, N, K, E, R)."""

LARGE, SMALL, FEW = range(3)
# for which rules: power of two alone, or both
SIZES = [(("fprop", 4096, 512, 9, 5120), LARGE), (("dgrad", 512, 4096, 9, 5120), LARGE),
         (("fprop", 4096, 640, 9, 5120), SMALL), (("dgrad", 640, 4096, 9, 5120), SMALL),
         (("fprop", 512, 1024, 9, 1536), FEW), (("dgrad", 1024, 512, 9, 1536), FEW),
         (("wgrad", 2048, 2048, 24, 10240), LARGE), (("wgrad", 256, 384, 9, 5120), SMALL)]

# Segments of rows, the expert in the middle of each always of 3 blocks: alone, among others, behind long ones.
MIDDLE = 384


def spreads(E, R):
    e, rest = E // 2, R - MIDDLE
    even = rest // (E - 1) // 128 * 128
    alone = [0] * E
    among = [even] * E
    behind = [0] * E
    behind[0], behind[E - 1] = rest // 256 * 128, 128
    some = [128 * (i % 3) for i in range(E)]
    while sum(some) > rest:
        some[some.index(max(some))] -= 128
    lists = [alone, among, behind, some]
    for lengths in lists:
        lengths[e] = MIDDLE
        assert sum(lengths) <= R
    return e, lists
