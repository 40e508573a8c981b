"""Sizes that reach each kernel of the operators of include/fp8moe.h once:
test_moe_paths.py checks on the host that they do, by the library's own rules;
the GPU tests run them."""
import numpy as np

# (T, H, I, E, k) of the mixture's wide kernels: few and many workgroups, one, two and four tiles of rows
WIDE = [(256, 384, 384, 86, 8), (100, 384, 384, 86, 8), (100, 384, 384, 64, 8), (200, 384, 384, 64, 8),
        (200, 256, 256, 64, 8), (40, 384, 384, 86, 8), (40, 640, 128, 86, 8)]
# of the narrow gate/up with several columns to a workgroup
NARROW = [(8, 256, 512, 128, 16), (4, 256, 896, 64, 16)]
# (M, N, K) of fp8_linear above FP8_LINEAR_FP32_ROWS: the wide kernel with four slots and with two, over more blocks than
# it keeps scales of at a time, columns that are and are not a multiple of eight, more rows than columns
LINEAR_WIDE = [(400, 4096, 4224), (700, 4096, 4224), (520, 3200, 8448), (3400, 640, 4224)]
# every tile of the other kernel
LINEAR_TILES = [(129, 384, 14720), (129, 768, 7424), (129, 1536, 4096), (200, 2048, 4096), (333, 2048, 2048),
                (200, 6144, 1152), (200, 5120, 1152)]
# either GEMM, and rows beyond it
LINEAR_GEMM = [(4133, 4096, 512), (10500, 4096, 640)]


def uneven_ids(T, E, k, seed):
    """A choice in which experts have from none to 80 rows, at and next to every
    border of the tiles, and the rest an even share; places left over are -1."""
    counts = [c for c in (0, 1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 80) if c <= T]
    share = (T * k - sum(counts)) // (E - len(counts))
    counts += [min(share, T)] * (E - len(counts))
    rng = np.random.default_rng(seed)
    ids, used, at = np.full((T, k), -1, np.int32), np.zeros(T, np.int64), 0
    for e, c in zip(rng.permutation(E), counts):
        for t in (at + np.arange(c)) % T:
            ids[t, used[t]] = e
            used[t] += 1
        at += c
    return rng.permuted(ids, axis=1)[rng.permutation(T)]
