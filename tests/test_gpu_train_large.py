"""The operators of include/fp8train.h at the sizes where another path or index
takes over, on the GPU: products of more tiles than workgroups, of hundreds of
experts, of reductions, columns and rows past each kernel's limit (whole numbers,
whose sums are exact in any order, against 64 bits), and buffers whose elements
pass 32 bits (rows that repeat, against the same call on one period, every
element)."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import train_cases
import train_ref
from blockwise_fp8_linear_amd import synth
from gpu_util import dev, dev_bf16, host, require_gpu

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
MODES = pytest.mark.parametrize("mode", [POW2, FP32])
WAYS = pytest.mark.parametrize("way", ["fprop", "dgrad", "wgrad"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _release():
    yield
    import torch
    torch.cuda.empty_cache()


# --------------------------------------------------------- grouped products --

class Whole:
    """Codes of -3 .. 3 and scales 1 .. 8 that change from group to group: whole numbers under either rule (a power of
    two is a scale of both), at most 9 * 2^6 a product.  With at most 2^14 of them to a sum every partial sum is a whole
    number below 2^24."""

    def __init__(self, E, N, K, lengths, behind, key, off=0):
        import torch
        self.g = torch.Generator("cuda").manual_seed(key)
        self.off = off      # words that the scales start behind an address of 16 bytes
        self.E, self.N, self.K, self.lengths = E, N, K, lengths
        self.offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        self.R = int(self.offsets[-1]) + behind
        self.w = self.codes(E * N, K)
        self.sw = self.scales(E * N // 128, K // 128)

    def codes(self, rows, cols):
        import torch
        v = torch.randint(-3, 4, (rows, cols), generator=self.g, device="cuda", dtype=torch.int8)
        return v.to(torch.bfloat16).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales(self, rows, cols):
        import torch
        s = torch.randint(0, 4, (rows, cols), generator=self.g, device="cuda").float().exp2()
        return torch.cat([s.new_zeros(self.off), s.view(-1)])[self.off:].view(rows, cols)

    def value(self, q, s, block=False):
        import torch
        v = q.view(torch.float8_e4m3fn).float()
        s = s.repeat_interleave(128, 1)
        return v * (s.repeat_interleave(128, 0) if block else s)

    def check(self, way, mode, experts=None):
        """Every element of `experts` (default all) against 64 bits; the rows of no segment as they were."""
        import torch
        E, N, K, R = self.E, self.N, self.K, self.R
        qw, sw = self.w.view(E, N, K), self.sw.view(E, N // 128, K // 128)
        off = dev(self.offsets)
        kw = dict(out_dtype=torch.float32, scale_mode=mode)
        experts = range(E) if experts is None else experts
        if way == "wgrad":
            a, sa, b, sb = self.codes(N, R), self.scales(N, R // 128), self.codes(K, R), self.scales(K, R // 128)
            out = fb.fp8_moe_gemm_wgrad(a, sa, b, sb, off, **kw)
            for e in experts:
                lo, hi = int(self.offsets[e]), int(self.offsets[e + 1])
                x = self.value(a[:, lo:hi], sa[:, lo // 128:hi // 128]).double()
                y = self.value(b[:, lo:hi], sb[:, lo // 128:hi // 128]).double()
                assert torch.equal(out[e].double(), x @ y.T.contiguous()), (way, e)
            return
        cols, red = (N, K) if way == "fprop" else (K, N)
        a, sa = self.codes(R, red), self.scales(R, red // 128)
        out = torch.full((R, cols), -0.5, device="cuda")
        (fb.fp8_moe_gemm_fprop if way == "fprop" else fb.fp8_moe_gemm_dgrad)(a, sa, qw, sw, off, out=out, **kw)
        for e in experts:
            lo, hi = int(self.offsets[e]), int(self.offsets[e + 1])
            w = self.value(qw[e], sw[e], True).double()
            x = self.value(a[lo:hi], sa[lo:hi]).double()
            assert torch.equal(out[lo:hi].double(), x @ (w.T.contiguous() if way == "fprop" else w)), (way, e)
        assert bool((out[int(self.offsets[-1]):] == -0.5).all())


@MODES
@pytest.mark.parametrize("i", range(len(train_cases.GROUPED)))
def test_grouped_every_kernel(i, mode):
    way, N, K, lengths, behind = train_cases.GROUPED[i]
    E = len(lengths)
    # 16512 products of 9 * 2^6 stay below 2^24
    Whole(E, N, K, lengths, behind, 100 + i).check(way, mode, None if E < 70 else [*range(0, E, 37), 1, 2, E // 2, E - 2, E - 1])


@MODES
@WAYS
def test_scales_off_16_bytes(way, mode):
    """Scales need 4 bytes of alignment only."""
    lengths = train_cases.some_lengths(12, 640)
    N, K = (512, 2048) if way == "dgrad" else (2048, 512)
    Whole(len(lengths), N, K, lengths, train_cases.whole(lengths), 99, off=1).check(way, mode)


@MODES
def test_wgrad_types_on_the_large_tiles(mode):
    """bf16, and what is added to, have the fp32 result."""
    import torch
    lengths = train_cases.some_lengths(64, 256)
    c = Whole(64, 1024, 1024, lengths, train_cases.whole(lengths), 98)
    a = c.codes(c.N, c.R), c.scales(c.N, c.R // 128), c.codes(c.K, c.R), c.scales(c.K, c.R // 128), dev(c.offsets)
    y = fb.fp8_moe_gemm_wgrad(*a, out_dtype=torch.float32, scale_mode=mode)
    assert torch.equal(fb.fp8_moe_gemm_wgrad(*a, scale_mode=mode), y.bfloat16())
    acc = torch.randn(y.shape, generator=c.g, device="cuda")
    want = acc + y
    fb.fp8_moe_gemm_wgrad(*a, out_dtype=torch.float32, out=acc, accumulate=True, scale_mode=mode)
    assert torch.equal(acc, want)


# ------------------------------------------------------- elements past 32 bits --

PERIOD, TIMES = 4096, 256
ROWS, COLS = PERIOD * TIMES, 4224      # 2^32 + 2^27 elements and more


def periodic(t, what):
    """A tensor of ROWS rows repeats `what`, of PERIOD rows."""
    for i in range(0, TIMES, 32):      # in pieces: a comparison makes a tensor of its own
        part = t[i * PERIOD:(i + 32) * PERIOD].view(32, PERIOD, -1)
        if not bool((part == what.view(1, PERIOD, -1)).all()):
            return False
    return True


def periodic_across(t, what):
    """The same of a transposed one, [cols][ROWS] (or its scales, ROWS / 128), in periods of what's columns."""
    n = what.shape[1]
    return all(bool((t[:, i * n:(i + 1) * n] == what).all()) for i in range(TIMES))


def rows_of(key, cols):
    return dev_bf16(synth.normal_bf16((PERIOD, cols), 1.0, 700 + key))


@MODES
@pytest.mark.parametrize("both", [False, True])
def test_gather_past_32_bits(both, mode):
    import torch
    x = rows_of(1, COLS)
    source = torch.arange(PERIOD, dtype=torch.int32, device="cuda").repeat(TIMES)
    got = fb.fp8_moe_gather(x, source, 1, transpose=both, scale_mode=mode)
    q, s = fb.fp8_quantize_rowgroup(x, scale_mode=mode)
    assert got[0].numel() > 2 ** 32 and periodic(got[0], q) and periodic(got[1], s)
    if both:
        qT, sT = fb.fp8_quantize_colgroup(x, scale_mode=mode)
        assert periodic_across(got[2], qT) and periodic_across(got[3], sT)


@pytest.mark.parametrize("weighted", [False, True])
def test_gather_in_the_order_of_tokens_past_32_bits(weighted):
    """Every choice of 65536 tokens once, spread over the rows."""
    import torch
    T, k = ROWS // 16, 16
    x = rows_of(2, COLS).repeat(T // PERIOD, 1)
    assert fb.fp8_moe_gather_workspace_size(T, COLS, ROWS, k) > 0
    order = torch.randperm(ROWS, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    w = torch.full((T, k), -2.0, device="cuda") if weighted else None
    q, s = fb.fp8_moe_gather(x, order.int(), k, weights=w)
    wq, ws = fb.fp8_quantize_rowgroup(x[:PERIOD] * -2 if weighted else x[:PERIOD])
    token = (order // k) % PERIOD
    for i in range(0, ROWS, 1 << 17):
        at = token[i:i + (1 << 17)]
        assert torch.equal(q[i:i + (1 << 17)], wq[at]) and torch.equal(s[i:i + (1 << 17)], ws[at])


@MODES
def test_gated_unit_and_turn_past_32_bits(mode):
    import torch
    gu, dh = rows_of(3, 2 * COLS), rows_of(4, COLS)
    small = fb.fp8_gated_forward(gu, scale_mode=mode)
    got = fb.fp8_gated_forward(gu.repeat(TIMES, 1), scale_mode=mode)
    assert got[0].numel() > 2 ** 32
    for g, w in zip(got, small):
        assert periodic(g, w)
    qc, sc = got[2:]
    wq, ws, wqT, wsT, wqhT, wshT = fb.fp8_gated_backward(dh, *small[2:], scale_mode=mode)
    q, s, qT, sT, qhT, shT = fb.fp8_gated_backward(dh.repeat(TIMES, 1), qc, sc, scale_mode=mode)
    assert periodic(q, wq) and periodic(s, ws)
    for g, w in ((qT, wqT), (sT, wsT), (qhT, wqhT), (shT, wshT)):
        assert periodic_across(g, w)
    del q, s, qT, sT, qhT, shT, got
    for g, w in zip(fb.fp8_requantize_colgroup(qc, sc, scale_mode=mode),
                    fb.fp8_requantize_colgroup(*small[2:], scale_mode=mode)):
        assert periodic_across(g, w)


def test_combine_and_its_gradient_past_32_bits():
    import torch
    T, k = PERIOD, 16
    z = rows_of(5, COLS).repeat(TIMES, 1)
    g = torch.Generator("cuda").manual_seed(6)
    rows = torch.randint(0, ROWS, (T, k), generator=g, device="cuda").int()
    rows[0], rows[-1] = ROWS - 1, ROWS
    w = torch.randn((T, k), generator=g, device="cuda")
    dy = rows_of(6, COLS)
    compact = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k).clone()
    compact[-1] = -1
    zc = z[rows.clamp(max=ROWS - 1).long().view(-1)]
    source = torch.full((ROWS,), -1, dtype=torch.int32, device="cuda")
    source[-T * k:] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    assert torch.equal(fb.fp8_moe_combine(z, rows, w), fb.fp8_moe_combine(zc, compact, w))
    q, s, qT, sT, dw = fb.fp8_moe_combine_backward(dy, z, rows, source, w)
    wq, ws, wqT, wsT, wdw = fb.fp8_moe_combine_backward(dy, zc, compact, source[-T * k:].contiguous(), w)
    assert torch.equal(dw, wdw) and bool((dw[-1] == 0).all())
    n = T * k
    for got, want in ((q, wq), (s, ws)):
        assert torch.equal(got[-n:], want) and bool((got[:-n] == (0 if got is q else 1)).all())
    assert torch.equal(qT[:, -n:], wqT) and torch.equal(sT[:, -n // 128:], wsT)


@MODES
def test_products_past_32_bits(mode):
    """1024 experts of a quarter of a period each: segment e holds the rows of segment e % 4."""
    import torch
    E, N, each = 1024, 128, PERIOD // 4
    x, dy = rows_of(7, COLS), rows_of(8, N)
    ends = torch.arange(0, ROWS + 1, each, dtype=torch.int32, device="cuda")
    qw, _, sw = fb.fp8_quantize_block(dev_bf16(synth.normal_bf16((4 * N, COLS), 0.02, 709)), transpose=False,
                                      scale_mode=mode)
    qw, sw = qw.view(4, N, COLS), sw.view(4, N // 128, COLS // 128)
    kw = dict(out_dtype=torch.float32, scale_mode=mode)
    for f, v, width in ((fb.fp8_moe_gemm_fprop, x, N), (fb.fp8_moe_gemm_dgrad, dy, COLS)):
        q, s = fb.fp8_quantize_rowgroup(v, scale_mode=mode)
        want = f(q, s, qw, sw, ends[:5], **kw)
        got = f(q.repeat(TIMES, 1), s.repeat(TIMES, 1), qw.repeat(TIMES, 1, 1), sw.repeat(TIMES, 1, 1), ends, **kw)
        assert got.shape == (ROWS, width) and periodic(got, want)
        del got
    a, b = fb.fp8_quantize_colgroup(dy, scale_mode=mode), fb.fp8_quantize_colgroup(x, scale_mode=mode)
    want = fb.fp8_moe_gemm_wgrad(*a, *b, ends[:5], **kw)
    got = fb.fp8_moe_gemm_wgrad(*(t.repeat(1, TIMES) for t in a + b), ends, **kw)
    for e in range(0, E, 4):
        assert torch.equal(got[e:e + 4], want), e


def test_sort_of_millions_of_choices():
    T, E, k = (1 << 20) + 37, 61, 4
    rng = synth.rng_for(712)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    R = fb.fp8_moe_sorted_rows(T, E, k)
    rows, source, offsets = (host(t) for t in fb.fp8_moe_sort(dev(ids), E))
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    first = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)])
    assert np.array_equal(offsets, first)
    want = np.full(R, -1, np.int32)
    at = np.concatenate([first[e] + np.arange(counts[e]) for e in range(E)])
    want[at] = order[:at.size]
    back = np.full(T * k, -1, np.int32)
    back[order[:at.size]] = at
    assert np.array_equal(source, want) and np.array_equal(rows.reshape(-1), back)


@pytest.mark.parametrize("T,E,k,H", [(4100, 9, 2, 1152), (4096, 30, 11, 128), (5000, 4, 3, 640)])
def test_weights_gradient_of_many_tokens(T, E, k, H):
    """A wave a token."""
    rng = synth.rng_for(713, T)
    R = fb.fp8_moe_sorted_rows(T, E, k)
    rows, source, _ = train_ref.sort(rng.integers(-1, E + 1, (T, k)).astype(np.int32), E, R)
    z, dy = synth.normal_bf16((R, H), 1.0, 714, T), synth.normal_bf16((T, H), 1.0, 715, T)
    w = rng.standard_normal((T, k)).astype(np.float32)
    dw = fb.fp8_moe_combine_backward(dev_bf16(dy), dev_bf16(z), dev(rows), dev(source), dev(w))[4]
    ref, bound = train_ref.dweights(train_ref.f64(dy), train_ref.f64(z), rows)
    assert np.all(np.abs(host(dw) - ref) <= bound)
