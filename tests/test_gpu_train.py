"""The operators of include/fp8train.h on the GPU, each against its 64-bit
reference (tests/train_ref.py): order, codes and scales of what is only moved or
requantized bit for bit, sums within the derived bounds, quantized results within
what either side of a rounding border gives; and what has to stay as it was."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import oracle
import train_ref
from blockwise_fp8_linear_amd import synth
from gpu_util import bf16_rne_np, check_f32, dev, dev_bf16, host, require_gpu
from train_ref import f64

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
MODES = pytest.mark.parametrize("mode", [POW2, FP32])
EMPTY = 0xA5    # what buffers hold before a call


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def codes_buffer(rows, cols, extra=0):
    """A code buffer of EMPTY bytes whose rows are `extra` bytes longer than they say."""
    import torch
    return torch.full((rows, cols + extra), EMPTY, dtype=torch.uint8, device="cuda")[:, :cols]


def scales_buffer(rows, cols):
    import torch
    return torch.full((rows, cols), -7.0, device="cuda")


def activations(M, K, key, ld=None):
    """bf16 bits with outlier channels, a row of zeros and tiny values; a device tensor whose rows are ld apart."""
    import torch
    bits = synth.normal_bf16((M, K), 1.0, 501, key)
    v = f64(bits)
    v[:, :: 97] *= 30.0
    if M > 2:
        v[1] = 0.0
        v[2] *= 2.0 ** -120
    bits = oracle.bf16_rne(v.astype(np.float32))
    t = dev_bf16(bits)
    if ld:
        wide = torch.full((M, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :K] = t
        t = wide[:, :K]
    return bits, t


def expect_rows(q, s, bits, mode, used):
    """Row groups of `bits` up to row `used`, what was there behind it."""
    oq, os = oracle.quantize_rowgroup(np.ascontiguousarray(bits), mode=mode)
    q, s = host(q), host(s)
    assert np.array_equal(q[:used], oq[:used]) and np.array_equal(s[:used], os[:used])
    assert (q[used:] == EMPTY).all() and (s[used:] == -7.0).all()


def expect_cols(qT, sT, bits, mode, used):
    oq, os = oracle.quantize_colgroup(np.ascontiguousarray(bits), mode=mode)
    qT, sT, g = host(qT), host(sT), -(-used // 128)
    assert np.array_equal(qT[:, :g * 128], oq[:, :g * 128]) and np.array_equal(sT[:, :g], os[:, :g])
    assert (qT[:, g * 128:] == EMPTY).all() and (sT[:, g:] == -7.0).all()


def limit(n):
    import torch
    return torch.tensor([n], dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------- sort --

def choice(T, E, k, kind, rng):
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    if kind == "odd":           # padding, ids that are no expert, the same id twice
        ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
        ids[rng.random((T, k)) < 0.05] = 2 ** 31 - 1
        ids[rng.random((T, k)) < 0.05] = -2 ** 31
        return ids
    p = rng.random(E) ** 3 + 1e-3
    return rng.choice(E, (T, k), p=p / p.sum()).astype(np.int32)


@pytest.mark.parametrize("T,E,k,kind", [
    (1, 1, 1, "even"), (1, 8, 2, "odd"), (5, 3, 3, "one"), (5, 3, 2, "none"), (64, 1, 1, "even"), (127, 2, 1, "one"),
    (128, 2, 1, "one"), (129, 2, 1, "one"), (511, 6, 2, "odd"), (1024, 60, 4, "odd"), (1025, 60, 4, "odd"),
    (1500, 1024, 16, "even"), (4095, 60, 4, "one"), (4096, 1024, 2, "odd"), (2731, 513, 3, "even"), (16384, 128, 8, "even"),
    (33000, 9, 8, "odd"), (20000, 1024, 16, "even"), (20000, 600, 16, "none")])
def test_sort(T, E, k, kind):
    import torch
    ids = choice(T, E, k, kind, synth.rng_for(31, T, E))
    R = fb.fp8_moe_sorted_rows(T, E, k)
    assert R == train_ref.sorted_rows(T, E, k)
    want = train_ref.sort(ids, E, R)
    for _ in range(2):
        room = [torch.full((n + 64,), -77, dtype=torch.int32, device="cuda") for n in (T * k, R, E + 1)]
        got = fb.fp8_moe_sort(dev(ids), E, rows=room[0][:T * k].view(T, k), source=room[1][:R], offsets=room[2][:E + 1])
        for g, w, r in zip(got, want, room):
            assert np.array_equal(host(g), w)
            assert bool((r[w.size:] == -77).all()), "wrote behind an output"


# ------------------------------------------------------------------- gather --

@MODES
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,E,k,H,ld,extra", [(1, 4, 1, 128, None, 0), (7, 3, 2, 640, 648, 16), (300, 5, 3, 256, None, 0),
                                              (200, 2, 2, 2048, 4096, 64)])
def test_gather(T, E, k, H, ld, extra, weighted, both, mode):
    rng = synth.rng_for(32, T, H)
    ids = choice(T, E, k, "odd", rng)
    R = fb.fp8_moe_sorted_rows(T, E, k)
    _, source, offsets = train_ref.sort(ids, E, R)
    bits, x = activations(T, H, T, ld)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    used = int(offsets[-1])
    out = dict(q=codes_buffer(R, H, extra), s=scales_buffer(R, H // 128))
    if both:
        out.update(qT=codes_buffer(H, R, extra), sT=scales_buffer(H, R // 128))
    r = fb.fp8_moe_gather(x, dev(source), k, used=limit(used), weights=None if w is None else dev(w), transpose=both,
                          scale_mode=mode, **out)
    rows = train_ref.gathered(bits, source, k, w)
    expect_rows(r[0], r[1], rows, mode, used)
    if both:
        expect_cols(r[2], r[3], rows, mode, used)


@pytest.mark.parametrize("used", [-5, 0, 1, 128, 129, 100000, None])
def test_gather_used_and_sources_of_no_choice(used):
    """`used` outside the buffer counts as its nearer end; a source that is no choice is a row of zeros."""
    T, k, H, R = 6, 2, 256, 384
    bits, x = activations(T, H, 3)
    source = synth.rng_for(33).integers(0, T * k, R).astype(np.int32)
    source[::3], source[1], source[7] = -1, T * k, 2 ** 31 - 1
    source[5] = -2 ** 31
    rows = train_ref.gathered(bits, source, k)
    end = R if used is None else -(-min(max(used, 0), R) // 128) * 128
    for both in (False, True):
        out = dict(q=codes_buffer(R, H), s=scales_buffer(R, H // 128))
        if both:
            out.update(qT=codes_buffer(H, R), sT=scales_buffer(H, R // 128))
        r = fb.fp8_moe_gather(x, dev(source), k, used=None if used is None else limit(used), transpose=both, **out)
        expect_rows(r[0], r[1], rows, POW2, end)
        if both:
            expect_cols(r[2], r[3], rows, POW2, end)


@MODES
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,E,k,H,part", [(4000, 20, 16, 1408, 1.0), (2100, 100, 14, 2176, 0.7)])
def test_gather_in_the_order_of_tokens(T, E, k, H, part, weighted, mode):
    """Sizes that are gathered in the order of their tokens; a device count that ends inside a run's rows and in padding,
    sources of no choice, and a source that stands in many rows."""
    rng = synth.rng_for(36, T, H)
    R = fb.fp8_moe_sorted_rows(T, E, k)
    assert fb.fp8_moe_gather_workspace_size(T, H, R, k) > 0
    _, source, offsets = train_ref.sort(choice(T, E, k, "odd", rng), E, R)
    source[rng.integers(0, R, 200)] = 5
    source[rng.integers(0, R, 50)] = [-7, T * k, 2 ** 31 - 1, -2 ** 31, -1] * 10
    bits, x = activations(T, H, T, H + 8)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    used = int(offsets[-1] * part) // 128 * 128
    q, s = fb.fp8_moe_gather(x, dev(source), k, used=limit(used), weights=None if w is None else dev(w),
                             q=codes_buffer(R, H, 16), s=scales_buffer(R, H // 128), scale_mode=mode)
    expect_rows(q, s, train_ref.gathered(bits, source, k, w), mode, used)


def groups_of_every_quotient():
    """bf16 bits [groups, 128]: for each mantissa of the amax, elements of every mantissa and sign in 20 octaves below it
    (the quotient's rounding depends on the mantissas alone), and for every exponent of the amax some of them."""
    rows = []
    for m in range(128):
        top = (127 << 7) | m
        rest = np.arange(top - 20 * 128, top + 1)
        rest = np.concatenate([rest, rest | 0x8000, [0, 0x8000]])
        rest = np.concatenate([rest, np.zeros(-rest.size % 127, rest.dtype)]).reshape(-1, 127)
        rows.append(np.concatenate([np.full((rest.shape[0], 1), top), rest], 1))
    rng = synth.rng_for(38)
    top = np.arange(0, 0x7F80, 37)
    rest = np.maximum(top[:, None] - rng.integers(0, 2500, (top.size, 127)), 0) | (rng.integers(0, 2, (top.size, 127)) << 15)
    rows.append(np.concatenate([top[:, None], rest], 1))
    return np.concatenate(rows).astype(np.uint16)


def test_short_quotient_gives_the_rule():
    """The amax / 448 codes of the kernels that take the short quotient (both forms of the gather, the gated unit's
    checkpoint) are the oracle's for every mantissa of the amax and the element."""
    x = groups_of_every_quotient()
    x = np.concatenate([x, np.zeros((-len(x) % 128, 128), np.uint16)])
    n = len(x)
    xt, source = dev_bf16(x), dev(np.arange(n, dtype=np.int32))
    q, s = fb.fp8_moe_gather(xt, source, 1, scale_mode=FP32)
    expect_rows(q, s, x, FP32, n)
    q, s, qT, sT = fb.fp8_moe_gather(xt, source, 1, transpose=True, scale_mode=FP32)
    expect_rows(q, s, x, FP32, n)
    expect_cols(qT, sT, x, FP32, n)
    across = np.ascontiguousarray(x.T)          # the groups down the columns of one block
    q, s, qT, sT = fb.fp8_moe_gather(dev_bf16(across), dev(np.arange(128, dtype=np.int32)), 1, transpose=True, scale_mode=FP32)
    expect_rows(q, s, across, FP32, 128)
    expect_cols(qT, sT, across, FP32, 128)
    gu = np.concatenate([x, x[::-1]], 1)
    _, _, qc, sc = fb.fp8_gated_forward(dev_bf16(gu), scale_mode=FP32)
    expect_rows(qc, sc, gu, FP32, n)


@MODES
def test_scale_of_every_amax(mode):
    """Every bf16 amax above zero, one to a group; waves hold groups of one size or of very different ones."""
    top = np.arange(1, 0x7F80, dtype=np.uint16)
    for order in (np.arange(top.size), synth.rng_for(39).permutation(top.size)):
        x = np.zeros((-(-top.size // 128) * 128, 128), np.uint16)
        x[:top.size, 3] = top[order]
        source = dev(np.arange(len(x), dtype=np.int32))
        q, s = fb.fp8_moe_gather(dev_bf16(x), source, 1, scale_mode=mode)
        expect_rows(q, s, x, mode, len(x))
        _, _, qT, sT = fb.fp8_moe_gather(dev_bf16(np.ascontiguousarray(x.T)), source[:128].contiguous(), 1, transpose=True,
                                         scale_mode=mode)
        expect_cols(qT, sT, np.ascontiguousarray(x.T), mode, 128)


@MODES
def test_values_that_are_not_finite(mode):
    """Codes and scales of the library's own quantizers, NaN and infinities in some groups and none in others."""
    import torch
    x = f64(activations(256, 384, 90)[0])
    x[3, 5], x[40, 200], x[41, 300], x[130:140, 7] = np.nan, np.inf, -np.inf, np.nan
    xt = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    want = fb.fp8_quantize_rowgroup(xt, scale_mode=mode) + fb.fp8_quantize_colgroup(xt, scale_mode=mode)
    source = dev(np.arange(256, dtype=np.int32))
    got = fb.fp8_moe_gather(xt, source, 1, transpose=True, scale_mode=mode)
    assert all(torch.equal(g.view(torch.uint8) if g.dtype is torch.uint8 else g.view(torch.int32),
                           w.view(torch.uint8) if w.dtype is torch.uint8 else w.view(torch.int32)) for g, w in zip(got, want))
    one = fb.fp8_moe_gather(xt, source, 1, scale_mode=mode)
    assert torch.equal(one[0], want[0]) and torch.equal(one[1].view(torch.int32), want[1].view(torch.int32))


# ------------------------------------------------------------------ combine --

def combine_case(T, E, k, H, ld=None):
    import torch
    rng = synth.rng_for(34, T, H, k)
    ids = choice(T, E, k, "odd", rng)
    R = fb.fp8_moe_sorted_rows(T, E, k)
    rows, source, offsets = train_ref.sort(ids, E, R)
    z = synth.normal_bf16((R, H), 1.0, 35, T)
    zt = torch.full((R, ld or H), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :H]
    live = source >= 0
    zt[dev(np.nonzero(live)[0])] = dev_bf16(z[live])       # what no choice stands in is NaN, and not read
    w = rng.standard_normal((T, k)).astype(np.float32)
    return rows, source, offsets, f64(z), zt, w, R


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,E,k,H,ld", [(1, 2, 1, 128, None), (9, 4, 2, 640, 704), (130, 40, 16, 384, None),
                                        (257, 12, 9, 2048, None), (65, 8, 8, 8320, None)])
def test_combine(T, E, k, H, ld, weighted):
    import torch
    rows, _, _, z, zt, w, R = combine_case(T, E, k, H, ld)
    rows = rows.copy()
    if T > 3:
        rows[2, 0], rows[3, 0] = R, -2 ** 31        # no rows of the buffer
    y, bound = train_ref.combine(z, rows, w if weighted else None)
    args = (zt, dev(rows), dev(w) if weighted else None)
    got = torch.full((T + 1, H), 5.0, device="cuda")
    fb.fp8_moe_combine(*args, out_dtype=torch.float32, out=got[:T])
    assert bool((got[T] == 5.0).all())
    assert np.all(np.abs(host(got[:T]) - y) <= bound)
    nothing = ((rows < 0) | (rows >= R)).all(1)
    assert (host(got[:T])[nothing] == 0).all()
    b = fb.fp8_moe_combine(*args)
    assert np.array_equal(host(b), bf16_rne_np(host(got[:T])))
    acc = torch.randn((T, H), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    want = acc + got[:T]
    fb.fp8_moe_combine(*args, out_dtype=torch.float32, out=acc, accumulate=True)
    assert torch.equal(acc, want)


@MODES
@pytest.mark.parametrize("T,E,k,H,ld", [(1, 2, 1, 128, None), (9, 4, 2, 640, 704), (130, 40, 16, 384, None),
                                        (200, 6, 3, 2176, None)])
def test_combine_backward(T, E, k, H, ld, mode):
    import torch
    rows, source, offsets, z, zt, w, R = combine_case(T, E, k, H, ld)
    bits, dy = activations(T, H, 8 + T, ld)
    used = int(offsets[-1])
    out = dict(q=codes_buffer(R, H), s=scales_buffer(R, H // 128), qT=codes_buffer(H, R), sT=scales_buffer(H, R // 128))
    room = torch.full((T + 1, k), 5.0, device="cuda")
    q, s, qT, sT, dw = fb.fp8_moe_combine_backward(dy, zt, dev(rows), dev(source), dev(w), used=limit(used),
                                                   dweights=room[:T], scale_mode=mode, **out)
    want = train_ref.gathered(bits, source, k, w)
    expect_rows(q, s, want, mode, used)
    expect_cols(qT, sT, want, mode, used)
    ref, bound = train_ref.dweights(f64(bits), z, rows)
    assert np.all(np.abs(host(dw) - ref) <= bound)
    assert (host(dw)[rows < 0] == 0).all() and bool((room[T] == 5.0).all())


# -------------------------------------------------------------- gated unit --

def check_between(q, s, value, err, mode, used):
    """Row-group codes of bf16(value), known to +-err, up to row `used`."""
    q, s = host(q), host(s)
    ref, off = train_ref.quantize_between(value, err, mode)
    got = train_ref.dequant(q[:used], s[:used])
    assert np.all(np.abs(got - ref[:used]) <= off[:used])
    return q, s


@MODES
@pytest.mark.parametrize("M,I,ld,extra,used", [(1, 128, None, 0, None), (3, 384, 800, 16, None), (130, 768, None, 0, None),
                                               (200, 256, None, 0, 77), (64, 256, None, 0, 0), (333, 2048, 4104, 0, 332)])
def test_gated_forward(M, I, ld, extra, used, mode):
    bits, gu = activations(M, 2 * I, 40 + M, ld)
    out = dict(q=codes_buffer(M, I, extra), s=scales_buffer(M, I // 128), qc=codes_buffer(M, 2 * I, extra),
               sc=scales_buffer(M, 2 * I // 128))
    n = M if used is None else used
    args = dict(used=None if used is None else limit(used), scale_mode=mode)
    q, s, qc, sc = fb.fp8_gated_forward(gu, **args, **out)
    expect_rows(qc, sc, bits, mode, n)
    h, err = train_ref.gated(f64(bits[:, :I]), f64(bits[:, I:]))
    q, s = check_between(q, s, h, err, mode, n)
    assert (q[n:] == EMPTY).all() and (s[n:] == -7.0).all()
    q2, s2 = fb.fp8_gated_forward(gu, checkpoint=False, **args)
    assert np.array_equal(host(q2)[:n], q[:n]) and np.array_equal(host(s2)[:n], s[:n])


@MODES
@pytest.mark.parametrize("M,I,ld,extra,used", [(128, 128, None, 0, None), (384, 256, 264, 16, 200), (256, 640, None, 0, 0),
                                               (2048, 1024, None, 0, None), (256, 2048, None, 0, 256)])
def test_gated_backward(M, I, ld, extra, used, mode):
    bits, gu = activations(M, 2 * I, 50 + M)
    _, _, qc, sc = fb.fp8_gated_forward(gu, scale_mode=mode)
    dbits, dh = activations(M, I, 51 + M, ld)
    out = dict(q=codes_buffer(M, 2 * I, extra), s=scales_buffer(M, 2 * I // 128), qT=codes_buffer(2 * I, M, extra),
               sT=scales_buffer(2 * I, M // 128), qhT=codes_buffer(I, M, extra), shT=scales_buffer(I, M // 128))
    n = M if used is None else -(-used // 128) * 128
    q, s, qT, sT, qhT, shT = fb.fp8_gated_backward(dh, qc, sc, used=None if used is None else limit(used),
                                                   scale_mode=mode, **out)
    kept = f64(train_ref.kept(host(qc), host(sc)))
    g, u = kept[:, :I], kept[:, I:]
    (dg, edg), (du, edu) = train_ref.gated_backward(g, u, f64(dbits))
    d, ed = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)
    q, s = check_between(q, s, d, ed, mode, n)
    assert (q[n:] == EMPTY).all() and (s[n:] == -7.0).all()
    if n:
        for qt, st, v, e in ((qT, sT, d, ed), (qhT, shT, *train_ref.gated(g, u))):
            ref, off = train_ref.quantize_between(np.ascontiguousarray(v[:n].T), np.ascontiguousarray(e[:n].T), mode)
            got = train_ref.dequant(host(qt)[:, :n], host(st)[:, :n // 128])
            assert np.all(np.abs(got - ref) <= off)
    for qt, st in ((qT, sT), (qhT, shT)):
        assert (host(qt)[:, n:] == EMPTY).all() and (host(st)[:, n // 128:] == -7.0).all()


@MODES
def test_gated_exact_where_the_sigmoid_is(mode):
    """|g| >= 160: the sigmoid is 1 or 0 in fp32, so h = g u or 0, du = dh g or 0, dg = dh u or 0 -- one product each
    (exact in fp32: 8 bits times 8), and every code has to be the oracle's."""
    M, I = 256, 384
    rng = synth.rng_for(61)
    g = rng.choice([160.0, -192.0, 1024.0, -20000.0, 224.0], (M, I)) * 2.0 ** rng.integers(0, 3, (M, 1))
    u = f64(synth.normal_bf16((M, I), 1.0, 62))
    gu = dev_bf16(oracle.bf16_rne(np.concatenate([g, u], 1).astype(np.float32)))
    q, s, qc, sc = fb.fp8_gated_forward(gu, scale_mode=mode)
    up = g > 0
    h = oracle.bf16_rne(np.where(up, g * u, 0.0).astype(np.float32))
    oq, os = oracle.quantize_rowgroup(h, mode=mode)
    assert np.array_equal(host(q) & 0x7F, oq & 0x7F) and np.array_equal(host(s), os)     # -0 where g < 0 < u
    dbits = synth.normal_bf16((M, I), 1e-2, 63)
    kept, dh = f64(train_ref.kept(host(qc), host(sc))), f64(dbits)
    g, u = kept[:, :I], kept[:, I:]
    assert np.array_equal(g > 0, up)
    d = np.concatenate([np.where(up, dh * u, 0.0), np.where(up, dh * g, 0.0)], 1)
    d, h = oracle.bf16_rne(d.astype(np.float32)), oracle.bf16_rne(np.where(up, g * u, 0.0).astype(np.float32))
    q, s, qT, sT, qhT, shT = (host(t) for t in fb.fp8_gated_backward(dev_bf16(dbits), qc, sc, scale_mode=mode))
    for got, want in ((q, oracle.quantize_rowgroup(d, mode=mode)), (qT, oracle.quantize_colgroup(d, mode=mode)),
                      (qhT, oracle.quantize_colgroup(h, mode=mode))):
        assert np.array_equal(got & 0x7F, want[0] & 0x7F)
    assert np.array_equal(s, oracle.quantize_rowgroup(d, mode=mode)[1])
    assert np.array_equal(sT, oracle.quantize_colgroup(d, mode=mode)[1])
    assert np.array_equal(shT, oracle.quantize_colgroup(h, mode=mode)[1])


@MODES
@pytest.mark.parametrize("M,C,extra,used", [(128, 128, 0, None), (384, 640, 16, 200), (2048, 1024, 0, None),
                                            (640, 256, 0, 0), (256, 384, 0, 256)])
def test_requantize(M, C, extra, used, mode):
    import torch
    bits, x = activations(M, C, 70 + M)
    wide = torch.zeros((M, C + extra), dtype=torch.uint8, device="cuda")
    q, s = fb.fp8_quantize_rowgroup(x, q=wide[:, :C], scale_mode=mode)
    if mode == POW2:
        s[3] = 2.0 ** 100          # scales of any power of two: groups of very different size share a column
    qT, sT = fb.fp8_requantize_colgroup(q, s, used=None if used is None else limit(used), qT=codes_buffer(C, M, extra),
                                        sT=scales_buffer(C, M // 128), scale_mode=mode)
    expect_cols(qT, sT, train_ref.kept(host(q), host(s)), mode, M if used is None else used)


# --------------------------------------------------------- grouped products --

LOADS = {"even": lambda E: [128] * E, "ragged": lambda E: [(0, 128, 640, 256, 0, 384)[e % 6] for e in range(E)],
         "one": lambda E: [0] * (E - 1) + [1152], "none": lambda E: [0] * E}


class Grouped:
    """Operands of the three products under one rule, quantized by the oracle, and their values in 64 bits."""

    def __init__(self, E, N, K, load, mode, whole=False, behind=256):
        rng = synth.rng_for(80, E, N, K)
        self.lengths = LOADS[load](E)
        self.offsets = np.concatenate([[0], np.cumsum(self.lengths)]).astype(np.int32)
        self.R = R = int(self.offsets[-1]) + behind
        self.E, self.N, self.K, self.mode = E, N, K, mode
        if whole:      # -3 .. 3 times powers of two that change from block to block
            def make(r, c):
                f = 2.0 ** rng.integers(0, 4, (-(-r // 128), -(-c // 128)))
                v = rng.integers(-3, 4, (r, c)) * np.repeat(np.repeat(f, 128, 0)[:r], 128, 1)[:, :c]
                return oracle.bf16_rne(v.astype(np.float32))
            x, dy, w = make(R, K), make(R, N), make(E * N, K)
        else:
            x, dy = synth.normal_bf16((R, K), 1.0, 81, K), synth.normal_bf16((R, N), 1e-3, 82, N)
            w = synth.normal_bf16((E * N, K), 0.02, 83, E)
        o = lambda f, v: f(v, mode=mode)  # noqa: E731
        self.qx, self.sx = o(oracle.quantize_rowgroup, x)
        self.qdy, self.sdy = o(oracle.quantize_rowgroup, dy)
        self.qxT, self.sxT = o(oracle.quantize_colgroup, x)
        self.qdyT, self.sdyT = o(oracle.quantize_colgroup, dy)
        qw, _, sw = oracle.quantize_block(w, transpose=False, mode=mode)
        self.qw, self.sw = qw.reshape(E, N, K), sw.reshape(E, N // 128, K // 128)

    def operands(self, way):
        a = {"fprop": (self.qx, self.sx, self.qw, self.sw), "dgrad": (self.qdy, self.sdy, self.qw, self.sw),
             "wgrad": (self.qdyT, self.sdyT, self.qxT, self.sxT)}[way]
        return [dev(t) for t in a] + [dev(self.offsets)]

    def shape(self, way):
        return {"fprop": (self.R, self.N), "dgrad": (self.R, self.K), "wgrad": (self.E, self.N, self.K)}[way]

    def want(self, way):
        """(the result in 64 bits, NaN where nothing is written; the sums of magnitudes)."""
        y = np.full(self.shape(way), 0.0 if way == "wgrad" else np.nan)
        size = np.zeros(self.shape(way))
        for e in range(self.E):
            lo, hi = self.offsets[e], self.offsets[e + 1]
            if way == "wgrad":
                if hi == lo:
                    continue
                a = train_ref.dequant(self.qdyT[:, lo:hi], self.sdyT[:, lo // 128:hi // 128])
                b = train_ref.dequant(self.qxT[:, lo:hi], self.sxT[:, lo // 128:hi // 128]).T
                at = e
            else:
                w = oracle.e4m3_decode(self.qw[e]) * np.repeat(np.repeat(self.sw[e].astype(np.float64), 128, 0), 128, 1)
                a = (train_ref.dequant(self.qx[lo:hi], self.sx[lo:hi]) if way == "fprop" else
                     train_ref.dequant(self.qdy[lo:hi], self.sdy[lo:hi]))
                b = w.T if way == "fprop" else w
                at = slice(lo, hi)
            y[at], size[at] = a @ b, np.abs(a) @ np.abs(b)
        return y, size

    def run(self, way, **kw):
        f = {"fprop": fb.fp8_moe_gemm_fprop, "dgrad": fb.fp8_moe_gemm_dgrad, "wgrad": fb.fp8_moe_gemm_wgrad}[way]
        return f(*self.operands(way), scale_mode=self.mode, **kw)


WAYS = pytest.mark.parametrize("way", ["fprop", "dgrad", "wgrad"])
SIZES = [(1, 128, 128, "even"), (3, 256, 384, "even"), (6, 384, 512, "ragged"), (7, 512, 1024, "ragged"),
         (12, 640, 256, "ragged"), (4, 1024, 512, "one"), (3, 256, 256, "none"), (40, 256, 512, "ragged")]


@MODES
@WAYS
@pytest.mark.parametrize("E,N,K,load", SIZES)
def test_grouped(E, N, K, load, way, mode):
    import torch
    c = Grouped(E, N, K, load, mode)
    y, size = c.want(way)
    out = torch.full(c.shape(way), float("nan"), device="cuda")
    c.run(way, out_dtype=torch.float32, out=out)
    got, live = host(out), ~np.isnan(y)
    assert np.array_equal(np.isnan(got), ~live), "rows of no segment are not written, the others are"
    if live.any() and size.any():
        check_f32(got[live], y[live], size[live], f"{way} {E} {N} {K} {load}")
        # the instruction's sums are off by 1.5e-5 .. 4.5e-5 of the result's norm; a term left out by 1 / sqrt(640) or more
        assert np.linalg.norm(got[live] - y[live]) <= 2e-4 * np.linalg.norm(y[live])
    b = torch.full(c.shape(way), float("nan"), dtype=torch.bfloat16, device="cuda")
    c.run(way, out=b)
    assert np.array_equal(host(b)[live], bf16_rne_np(got[live])) and bool(torch.equal(b.isnan(), out.isnan()))
    acc = torch.randn(c.shape(way), generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    want = torch.where(out.isnan(), acc, acc + out)
    c.run(way, out_dtype=torch.float32, out=acc, accumulate=True)
    assert torch.equal(acc, want)


@MODES
@WAYS
@pytest.mark.parametrize("E,N,K,load", [(6, 384, 512, "ragged"), (4, 512, 1024, "one"), (13, 256, 640, "ragged")])
def test_grouped_exact(E, N, K, load, way, mode):
    """Whole numbers under scales that change from block to block: at most 1280 products of 9 times 2^6, so that every
    partial sum is a whole number below 2^24 and the order cannot matter.  (Under the amax / 448 rule codes are not
    exact; there the result is only compared between calls that place the segments differently.)"""
    import torch
    c = Grouped(E, N, K, load, mode, whole=True)
    out = torch.full(c.shape(way), float("nan"), device="cuda")
    c.run(way, out_dtype=torch.float32, out=out)
    if mode == POW2:
        y, _ = c.want(way)
        assert np.array_equal(host(out), y.astype(np.float32), equal_nan=True)
    again = torch.full(c.shape(way), float("nan"), device="cuda")
    c.run(way, out_dtype=torch.float32, out=again)
    assert torch.equal(out.nan_to_num(7.0), again.nan_to_num(7.0))


@WAYS
def test_grouped_results_do_not_depend_on_the_other_experts(way):
    """An expert alone in its call has the bits that it has among others."""
    import torch
    c = Grouped(7, 512, 1024, "ragged", POW2)
    all_ = c.run(way, out_dtype=torch.float32)
    lo, hi = int(c.offsets[2]), int(c.offsets[3])
    ops = c.operands(way)
    if way == "wgrad":
        one = fb.fp8_moe_gemm_wgrad(ops[0][:, lo:hi].contiguous(), ops[1][:, lo // 128:hi // 128].contiguous(),
                                    ops[2][:, lo:hi].contiguous(), ops[3][:, lo // 128:hi // 128].contiguous(),
                                    dev(np.array([0, hi - lo], np.int32)), out_dtype=torch.float32)
        assert torch.equal(one[0], all_[2])
    else:
        f = fb.fp8_moe_gemm_fprop if way == "fprop" else fb.fp8_moe_gemm_dgrad
        one = f(ops[0][lo:hi], ops[1][lo:hi], ops[2][2:3], ops[3][2:3], dev(np.array([0, hi - lo], np.int32)),
                out_dtype=torch.float32)
        assert torch.equal(one, all_[lo:hi])


@WAYS
def test_grouped_odd_offsets_stay_inside(way):
    """Offsets outside the buffer or between multiples of 128 count as documented; descending ones touch nothing else."""
    import torch
    c = Grouped(4, 256, 512, "even", POW2, behind=0)
    ok = c.run(way, out_dtype=torch.float32)
    c.offsets = np.array([-300, 200, 257, 384 + 127, 99999], np.int32)      # 0, 128, 256, 384, 512
    assert torch.equal(c.run(way, out_dtype=torch.float32), ok)
    c.offsets = np.array([0, 512, 128, 128, 512], np.int32)
    room = torch.full((c.shape(way)[0] + 2, *c.shape(way)[1:]), -3.0, device="cuda")
    c.run(way, out_dtype=torch.float32, out=room[1:-1])
    assert bool((room[0] == -3.0).all()) and bool((room[-1] == -3.0).all())
