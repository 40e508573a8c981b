"""The one-pass kernels on tiles in blocks that the size does not fill, on the
GPU: whole calls against calls on a few rows, which take their tiles row band by
row band and are compared with the oracle elsewhere."""
import pytest

import blockwise_fp8_linear_amd as fb
import tile_cases
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
MODES = pytest.mark.parametrize("mode", [POW2, FP32])
SIZES = pytest.mark.parametrize("tiles", tile_cases.BLOCKED)
EMPTY = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _release():
    yield
    import torch
    torch.cuda.empty_cache()


def random(rows, cols, key):
    """bf16 rows of different sizes, a part of them zeros."""
    import torch
    g = torch.Generator("cuda").manual_seed(key)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.randint(-12, 3, (rows, 1), generator=g, device="cuda").float().exp2()
    x[::37] = 0
    return x.bfloat16()


def codes(rows, cols):
    import torch
    return (torch.full((rows, cols), EMPTY, dtype=torch.uint8, device="cuda"),
            torch.full((rows, cols // 128), -7.0, device="cuda"))


def limit(n):
    import torch
    return torch.tensor([n], dtype=torch.int32, device="cuda")


def compare(outs, piece, rows, used):
    """outs: [(codes, scales, transposed)] of a call on `rows` rows up to `used`; piece(lo, hi): those of a call on the
    rows lo .. hi - 1."""
    import torch
    step = 128 * tile_cases.PIECE
    for lo in range(0, used, step):
        hi = min(lo + step, used)
        for (q, s, across), (wq, ws) in zip(outs, piece(lo, hi)):
            if across:
                assert torch.equal(q[:, lo:hi], wq) and torch.equal(s[:, lo // 128:hi // 128], ws), (lo, hi)
            else:
                assert torch.equal(q[lo:hi], wq) and torch.equal(s[lo:hi], ws), (lo, hi)
    for q, s, across in outs:
        q, s = (q[:, used:], s[:, used // 128:]) if across else (q[used:], s[used:])
        assert bool((q == EMPTY).all()) and bool((s == -7.0).all()), "wrote behind the rows in use"


def in_use(rows):
    return rows, rows // 128 * 5 // 7 * 128


@MODES
@SIZES
def test_gated_backward(tiles, mode):
    M, I = 128 * tiles[0], 128 * tiles[1]
    _, _, qc, sc = fb.fp8_gated_forward(random(M, 2 * I, 1), scale_mode=mode)
    dh = random(M, I, 2)

    def piece(lo, hi):
        r = fb.fp8_gated_backward(dh[lo:hi], qc[lo:hi], sc[lo:hi], scale_mode=mode)
        return r[0:2], r[2:4], r[4:6]

    for used in in_use(M):
        (q, s), (qT, sT), (qhT, shT) = codes(M, 2 * I), codes(2 * I, M), codes(I, M)
        fb.fp8_gated_backward(dh, qc, sc, used=limit(used), q=q, s=s, qT=qT, sT=sT, qhT=qhT, shT=shT, scale_mode=mode)
        compare([(q, s, False), (qT, sT, True), (qhT, shT, True)], piece, M, used)


@MODES
@SIZES
def test_requantize(tiles, mode):
    M, C = 128 * tiles[0], 128 * tiles[1]
    q, s = fb.fp8_quantize_rowgroup(random(M, C, 3), scale_mode=mode)
    for used in in_use(M):
        qT, sT = codes(C, M)
        fb.fp8_requantize_colgroup(q, s, used=limit(used), qT=qT, sT=sT, scale_mode=mode)
        compare([(qT, sT, True)], lambda lo, hi: [fb.fp8_requantize_colgroup(q[lo:hi], s[lo:hi], scale_mode=mode)], M, used)


@MODES
@pytest.mark.parametrize("k", [1, 3])
@SIZES
def test_gather(tiles, k, mode):
    """Columns that are one XCD's for all rows (some k above 1) among them."""
    import torch
    R, H, T = 128 * tiles[0], 128 * tiles[1], 500
    x = random(T, H, 4)
    g = torch.Generator("cuda").manual_seed(5)
    source = torch.randint(-T * k // 9, T * k, (R,), generator=g, device="cuda").int()
    w = torch.randn((T, k), generator=g, device="cuda") if k > 1 else None

    def piece(lo, hi):
        r = fb.fp8_moe_gather(x, source[lo:hi].contiguous(), k, weights=w, transpose=True, scale_mode=mode)
        return r[:2], r[2:]

    for used in in_use(R):
        (q, s), (qT, sT) = codes(R, H), codes(H, R)
        fb.fp8_moe_gather(x, source, k, used=limit(used), weights=w, transpose=True, q=q, s=s, qT=qT, sT=sT, scale_mode=mode)
        compare([(q, s, False), (qT, sT, True)], piece, R, used)
