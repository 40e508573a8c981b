"""fp8_linear above FP8_LINEAR_FP32_ROWS rows: every kernel it has there
(test_moe_paths.py holds the sizes to that), by whole numbers under different
scales for every token and weight block, whose sums are exact on either matrix
instruction, and by the error's size against the result's."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import moe_cases
import moe_ref
import oracle
from blockwise_fp8_linear_amd import synth
from gpu_util import dev, dev_bf16, host, require_gpu

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("M,N,K", moe_cases.LINEAR_WIDE + moe_cases.LINEAR_TILES + moe_cases.LINEAR_GEMM)
def test_exact(M, N, K):
    """-3 .. 3 times a power of two that changes from token to token and from
    block to block: codes are exact, a block's sum is a whole number of at most
    1152 times its scales, and K 9 2^6 < 2^24 keeps every partial sum whole."""
    import torch
    assert K * 9 * 64 < 2 ** 24
    rng, nkb = synth.rng_for(91, M), K // 128
    m, n, b = np.arange(M)[:, None], np.arange(N)[:, None] // 128, np.arange(nkb)[None, :]
    x = (rng.integers(-3, 4, (M, nkb, 128)) * 2.0 ** ((m + 3 * b) % 4)[:, :, None]).reshape(M, K)
    w = (rng.integers(-3, 4, (N, nkb, 128)) * 2.0 ** ((2 * n + b) % 4)[:, :, None]).reshape(N, K)
    qw, _, sw = oracle.quantize_block(oracle.bf16_rne(w.astype(np.float32)), transpose=False)
    xt = dev_bf16(oracle.bf16_rne(x.astype(np.float32)))
    want = (x @ w.T).astype(np.float32)
    y = torch.full((M + 1, N), float("nan"), device="cuda")
    fb.fp8_linear(xt, dev(qw), dev(sw), out_dtype=torch.float32, out=y[:M])
    assert np.array_equal(host(y[:M]), want)
    assert bool(torch.isnan(y[M]).all()), "wrote past the last row"
    assert torch.equal(fb.fp8_linear(xt, dev(qw), dev(sw)), dev(want).bfloat16())


@pytest.mark.parametrize("M,N,K,mode", [(400, 4096, 4224, POW2), (700, 4096, 4224, POW2), (700, 4096, 4224, FP32),
                                        (520, 3200, 8448, FP32), (333, 2048, 2048, POW2), (200, 5120, 1152, FP32),
                                        (4133, 4096, 512, POW2), (2048, 4096, 2048, FP32)])
def test_error_is_small_against_the_result(M, N, K, mode):
    """The fp8 instruction's sums are off by 1.5e-5 of the result's norm.  Seven
    times that, per token: a product of average size left out of each sum would
    be 1 / sqrt(K) >= 1e-2 of it, a wrong scale more."""
    import torch
    x, w = synth.normal_bf16((M, K), 1.0, 92, M), synth.normal_bf16((N, K), 0.02, 93, N)
    qw, _, sw = oracle.quantize_block(w, transpose=False, mode=mode)
    y = host(fb.fp8_linear(dev_bf16(x), dev(qw), dev(sw), out_dtype=torch.float32, scale_mode=mode)).astype(np.float64)
    ref = moe_ref.dequant_rows(x, mode) @ moe_ref.dequant_block(qw, sw).T
    size = np.linalg.norm(ref, axis=1)
    off = np.linalg.norm(y - ref, axis=1) / size
    assert np.all(off <= 1e-4), float(off.max())
    if moe_cases.LINEAR_TILES.count((M, N, K)):  # on the bf16 instruction: fp32 sums
        _, bound = moe_ref.product(moe_ref.dequant_rows(x, mode), moe_ref.dequant_block(qw, sw))
        assert np.all(np.abs(y - ref) <= bound)
