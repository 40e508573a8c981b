"""Sizes, in tiles of 128, at which the one-pass kernels take their tiles in
blocks that the size does not fill (tests/test_tile_order.py checks that it does)."""

BLOCKED = [(30, 31),     # 2 x 4 blocks, rows and columns over
           (61, 15),     # 4 x 2
           (121, 5),     # one column of blocks, narrow
           (128, 8),     # whole blocks
           (320, 23)]    # 60 of 64 blocks
PIECE = 7                # row tiles of a call that does not
