"""Segments of experts for the grouped products' tests; tests/test_train_paths.py
checks that they reach every kernel."""


def some_lengths(E, each):
    """Segments around `each` rows with every remainder mod 256, every fourth without rows."""
    return [0 if e % 4 == 3 else max(0, each + 128 * ((e * 5) % 7 - 3)) for e in range(E)]


def rows(lengths, behind):
    return sum(lengths) + behind


def whole(lengths, behind=128):
    """`behind` such that the rows are a multiple of 512, as the sort's are."""
    return behind + -rows(lengths, behind) % 512


# (way, N, K, lengths, rows behind): whole numbers, at most 2^14 products of 9 * 2^6 a sum
GROUPED = []
for _cols, _red, _E, _each in ((2048, 512, 12, 640), (2048, 640, 12, 640), (2304, 512, 9, 1408), (2304, 384, 9, 1408),
                               (256, 1024, 40, 384)):
    _l = some_lengths(_E, _each)
    GROUPED += [("fprop", _cols, _red, _l, 256), ("dgrad", _red, _cols, _l, 256), ("wgrad", _cols, _red, _l, whole(_l))]
# Wgrad on the large tiles: several tiles a workgroup, more experts than are put in order, edges inside a tile
GROUPED += [("wgrad", 1024, 1024, _l, whole(_l)) for _l in (some_lengths(64, 256),)]
GROUPED += [("wgrad", 512, 512, _l, whole(_l)) for _l in (some_lengths(300, 384), [0] * 299 + [4096])]
GROUPED += [("wgrad", 1920, 1152, _l, whole(_l)) for _l in (some_lengths(32, 1920),)]
GROUPED += [("wgrad", 2048, 2048, _l, _b) for _l in ([1408] * 8,) for _b in (whole([1408] * 8), 128)]
# hundreds of experts
for _E in (255, 257, 1000, 1024):
    _l = [128 * (e % 3) for e in range(_E)]
    _l[-1], _l[_E // 2] = 384, 1152
    GROUPED += [(_w, 256, 128, _l, 128) for _w in ("fprop", "dgrad", "wgrad")]
# few rows
GROUPED += [("fprop", 640, 384, [128, 0, 256], 128), ("dgrad", 1152, 256, [128, 0, 256], 128),
            ("fprop", 256, 1024, [256, 128], 128), ("dgrad", 1024, 384, [256, 128], 128)]
# long reductions, many columns, more rows than 32-bit lane offsets take
GROUPED += [("fprop", 128, 16384, [128, 0, 384], 128), ("dgrad", 16512, 256, [256, 128], 128),
            ("fprop", 4096, 16384, [1024, 128], 128), ("fprop", 4096, 16512, [1024, 128], 128),
            ("fprop", (1 << 22) + 256, 128, [128, 256], 128), ("dgrad", 512, (1 << 22) + 128, [384], 128),
            ("wgrad", 128, 128, [4096] * 1024, 4096), ("wgrad", 1024, 1024, [4096] * 16, (1 << 22) - 4096 * 16 + 512)]
