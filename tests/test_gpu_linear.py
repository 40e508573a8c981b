"""fp8_linear against a 64-bit product of the oracle's quantized operands:
every token count where its launch changes, odd sizes, strides, both scale
rules, all output types."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import moe_ref
import oracle
from blockwise_fp8_linear_amd import synth
from gpu_util import RTOL, bf16_rne_np, dev, dev_bf16, host, require_gpu

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _run(M, N, K, mode, x=None, seed=0, ld=None):
    import torch
    x = synth.normal_bf16((M, K), 1.0, 60, seed, M) if x is None else x
    w = synth.normal_bf16((N, K), 0.02, 61, seed, N)
    qw, _, sw = oracle.quantize_block(w, transpose=False, mode=mode)
    wide = torch.full((M, ld or K), 1e30, device="cuda", dtype=torch.bfloat16)
    wide[:, :K] = dev_bf16(x)
    y = torch.full((M + 1, N), float("nan"), device="cuda", dtype=torch.float32)
    fb.fp8_linear(wide[:, :K], dev(qw), dev(sw), out_dtype=torch.float32, out=y[:M], scale_mode=mode)
    assert bool(torch.isnan(y[M]).all()), "wrote past the last row"
    return wide[:, :K], (dev(qw), dev(sw)), host(y[:M]), (moe_ref.dequant_rows(x, mode), moe_ref.dequant_block(qw, sw))


M_ALL = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 100, 127, 128, 129, 200, 255, 256, 257, 383, 513,
         700]
SHAPES = [(1, 128, 128), (5, 128, 1152), (3, 1152, 128), (16, 256, 2048), (1, 2048, 6144), (40, 384, 768),
          (7, 8192, 256), (20, 12288, 128), (33, 16384, 256), (64, 640, 384), (130, 8192, 128),
          (700, 8192, 128), (475, 8192, 256), (1100, 4096, 128), (2048, 2048, 128),
          (1500, 8192, 512), (1200, 8192, 512), (2300, 8192, 128), (513, 3328, 640), (128, 25600, 128),
          (9, 128, 2176), (77, 256, 2304), (65, 512, 13312), (200, 640, 8192), (333, 1152, 4224), (129, 2176, 5120),
          (1027, 384, 7680), (9, 65536, 256), (120, 24576, 384), (1600, 2048, 128), (1500, 1664, 256),
          (2100, 4096, 640), (3000, 3968, 128),
          (64, 2048, 6400), (200, 4096, 1152), (40, 12288, 128), (1230, 8192, 1024), (4, 6144, 256)]


@pytest.mark.parametrize("M,N,K,mode", [(m, 256, 384, POW2) for m in M_ALL] +
                         [(m, 384, 256, FP32) for m in M_ALL[::3]] +
                         [(*s, mode) for s in SHAPES for mode in (POW2, FP32)])
def test_linear(M, N, K, mode):
    import torch
    xt, w, y, (xd, wd) = _run(M, N, K, mode, ld=K + 40)
    ref, bound = moe_ref.product(xd, wd)
    if M > fb.FP8_LINEAR_FP32_ROWS:              # rows that go through the GEMMs are held to their gate
        bound = np.maximum(bound, RTOL * (np.abs(xd) @ np.abs(wd).T))
    err = np.abs(y - ref)
    assert np.all(err <= bound), float(np.max(err / bound))
    b = fb.fp8_linear(xt, *w, scale_mode=mode)
    assert np.array_equal(host(b), bf16_rne_np(y)), "bf16 is not the rounding of the fp32 result"
    acc = torch.ones((M, N), device="cuda")
    fb.fp8_linear(xt, *w, scale_mode=mode, out_dtype=torch.float32, out=acc, accumulate=True)
    assert np.array_equal(host(acc), (np.float32(1) + y).astype(np.float32))


def test_whole_numbers_are_exact():
    """Small whole numbers quantize losslessly: the product is exact."""
    import torch
    rng = synth.rng_for(62)
    for M in (1, 30, 64, 300):
        x, w = rng.integers(-15, 16, (M, 512)), rng.integers(-15, 16, (256, 512))
        qw, _, sw = oracle.quantize_block(oracle.bf16_rne(w.astype(np.float32)), transpose=False)
        y = fb.fp8_linear(dev_bf16(oracle.bf16_rne(x.astype(np.float32))), dev(qw), dev(sw), out_dtype=torch.float32)
        assert np.array_equal(host(y).astype(np.int64), x @ w.T), M


@pytest.mark.parametrize("mode", [POW2, FP32])
@pytest.mark.parametrize("M,N,K", [(3, 128, 512), (40, 128, 512), (100, 128, 512), (400, 4096, 512), (100, 128, 2176)])
def test_quantizes_as_the_quantizer(M, N, K, mode):
    """Groups of zeros, subnormals, huge values and outliers: with W = 1 at
    one place of each block row the output is the quantizer's code times its
    scale (times W's), which the fp32 sum leaves alone."""
    import torch
    x = synth.normal_bf16((M, K), 1.0, 63, M)
    x[0, :128] = 0                               # a group of +0
    x[1, 128:256] = 0x8000                       # -0
    x[2, :128] = synth.rng_for(64).integers(0, 0x80, 128).astype(np.uint16)       # subnormals
    x[M - 1, 256:384] = 0x7F7F                   # the largest finite
    x[M - 1, 300] = 1
    W = np.zeros((N, K), np.float32)
    at = synth.rng_for(65).integers(0, K, N)
    W[np.arange(N), at] = 1.0
    qw, _, sw = oracle.quantize_block(oracle.bf16_rne(W), transpose=False, mode=mode)
    y = host(fb.fp8_linear(dev_bf16(x), dev(qw), dev(sw), out_dtype=torch.float32, scale_mode=mode)).astype(np.float64)
    # the largest bf16, (2 - 2^-7) 2^127, rounds to the code 256 at the scale 2^120: 2^128, which fp32 holds as infinity
    want = (moe_ref.dequant_rows(x, mode) @ moe_ref.dequant_block(qw, sw).T)
    over = np.abs(want) >= 2.0 ** 128
    assert np.array_equal(np.isinf(y), over)
    y, want = np.where(over, 0, y), np.where(over, 0, want)
    # one product per output: the scale product's rounding and its own (an underflow is off by the least subnormal)
    assert np.all(np.abs(y - want) <= 4 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149 * 448 * 448)


def test_many_rows_of_few_columns():
    """More groups than one launch of the quantizer has places for: the first
    and the last rows against the product, and the last as a call of their
    own."""
    import torch
    M, N, K = 45000, 128, 4096
    x = synth.normal_bf16((64, K), 1.0, 70)
    w = synth.normal_bf16((N, K), 0.02, 71)
    qw, _, sw = oracle.quantize_block(w, transpose=False)
    xt = torch.zeros((M, K), device="cuda", dtype=torch.bfloat16)
    xt[:32], xt[-32:] = dev_bf16(x[:32]), dev_bf16(x[32:])
    y = fb.fp8_linear(xt, dev(qw), dev(sw), out_dtype=torch.float32)
    assert not bool(y[32:-32].any())
    xd, wd = moe_ref.dequant_rows(x, POW2), moe_ref.dequant_block(qw, sw)
    ref, _ = moe_ref.product(xd, wd)
    bound = RTOL * (np.abs(xd) @ np.abs(wd).T)
    assert np.all(np.abs(np.concatenate([host(y[:32]), host(y[-32:])]) - ref) <= bound)


def test_two_threads_at_once():
    """Calls from two host threads, each on its own stream with its own
    workspaces, give what either gives alone."""
    import threading
    import torch
    E, H, I, k = 12, 256, 384, 3
    q1, _, s1 = fb.fp8_quantize_block(dev_bf16(synth.normal_bf16((E * 2 * I, H), 0.06, 72)), transpose=False)
    q2, _, s2 = fb.fp8_quantize_block(dev_bf16(synth.normal_bf16((E * H, I), 0.06, 73)), transpose=False)
    exps = (q1.view(E, 2 * I, H), s1.view(E, 2 * I // 128, H // 128), q2.view(E, H, I), s2.view(E, H // 128, I // 128))
    qw, _, sw = fb.fp8_quantize_block(dev_bf16(synth.normal_bf16((512, H), 0.06, 74)), transpose=False)
    wr = dev_bf16(synth.normal_bf16((E, H), 0.3, 75))
    xs = [dev_bf16(synth.normal_bf16((T, H), 1.0, 76, T)) for T in (3, 12, 60, 200)]

    def step(x):
        lg = fb.fp8_linear(x, qw, sw, out_dtype=torch.float32)
        ids, w = fb.fp8_moe_route(lg, 4)
        return [lg, ids, w, fb.fp8_moe_route_backward(lg, ids, w), fb.fp8_moe_layer(x, wr, *exps, k)]

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def run(order):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = [(i, step(xs[i])) for i in order]
                    torch.cuda.current_stream().synchronize()
                    bad.extend(i for i, g in got if not all(torch.equal(a, b) for a, b in zip(g, want[i])))
        except Exception as e:  # noqa: BLE001 -- reported by the test's own thread
            bad.append(e)

    threads = [threading.Thread(target=run, args=(o,)) for o in ([0, 1, 2, 3], [3, 1, 0, 2])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


def test_equals_the_quantizer_and_fprop():
    """Multiples of 128 rows that fill the GEMM's tiles are the library's own
    quantizer and GEMM, bit for bit."""
    import torch
    M, N, K = 4096, 2048, 512
    x, w = dev_bf16(synth.normal_bf16((M, K), 1.0, 66)), dev_bf16(synth.normal_bf16((N, K), 0.02, 67))
    qw, _, sw = fb.fp8_quantize_block(w, transpose=False)
    qx, sx = fb.fp8_quantize_rowgroup(x)
    assert torch.equal(fb.fp8_linear(x, qw, sw), fb.fp8_block_gemm_fprop(qx, sx, qw, sw))


def test_graph_and_stream():
    import torch
    for M in (2, 77, 300):
        x = dev_bf16(synth.normal_bf16((M, 256), 1.0, 68, M))
        qw, _, sw = fb.fp8_quantize_block(dev_bf16(synth.normal_bf16((384, 256), 0.02, 69)), transpose=False)
        ref = fb.fp8_linear(x, qw, sw)
        y = torch.empty_like(ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fb.fp8_linear(x, qw, sw, out=y)
        for _ in range(3):
            y.fill_(9.0)
            torch.randn(64, 64, device="cuda").sum()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ref)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        z = fb.fp8_linear(x, qw, sw, stream=s)
        s.synchronize()
        assert torch.equal(z, ref)
