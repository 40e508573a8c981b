"""Where 32 bits end, on the GPU.  The gated unit: a sigmoid below fp32's normal
range times values near its limit, and a product dh u past it whose gradient is not.
Against the formulas in 64 bits.  And the ends of the range of the amax / 448
quotients."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import oracle
import train_ref
from blockwise_fp8_linear_amd import synth
from gpu_util import dev, dev_bf16, host, require_gpu
from train_ref import U, f64

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
MODES = pytest.mark.parametrize("mode", [POW2, FP32])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def unit(g, u):
    """(h, bound) before its rounding to bf16.  e^-g's argument is rounded twice (the constant, the product), 2 |g| U of
    it; powers of two to one ulp (2 U), at most four of them; the sum and the quotient one rounding each; the two products
    and the rounding to fp32 (2^-149 where that is not normal) one each."""
    h = g * u / (1.0 + np.exp(-g))
    return h, (2 * np.abs(g) + 16) * U * np.abs(h) + 2.0 ** -149


def gradient(g, u, dh):
    """((dg, bound), (du, bound)): f = sig (1 + g (1 - sig)); sig is off by es, 1 - sig by as much and a rounding."""
    s = 1.0 / (1.0 + np.exp(-g))
    es = (2 * np.abs(g) + 16) * U * s
    f = s * (1.0 + g * (1.0 - s))
    ef = es * (1.0 + np.abs(g)) + s * (np.abs(g) * (es + 2 * U) + 3 * U * (1.0 + np.abs(g)))
    du, edu = unit(g, dh)
    return (dh * u * f, np.abs(dh * u) * ef + 4 * U * np.abs(dh * u * f) + 2.0 ** -149), (du, edu)


def expect(q, s, value, err, mode):
    ref, off = train_ref.quantize_between(value, err, mode)
    got = train_ref.dequant(host(q), host(s))
    assert np.isfinite(got).all() and np.all(np.abs(got - ref) <= off)
    return got


def signs(rng, shape):
    return rng.choice([-1.0, 1.0], shape)


# (least and greatest -g of a tile, u, dh)
TILES = [(88, 96, 3e38, 1.0), (96, 112, 1e38, 30.0), (120, 128, 3e38, 1e-3), (144, 160, 2e38, 1.0), (160, 168, 3e38, 1e6),
         (25, 32, 1e23, 1e19), (40, 48, 3e38, 1e13), (80, 87, 1e30, 1e20),
         (100, 108, 1.0, 3e38), (136, 144, 1e-6, 3e38)]


def tiles(key):
    """bf16 bits [128, 128 a tile] of g, u and dh."""
    rng = synth.rng_for(901, key)
    out = []
    for lo, hi, u, dh in TILES:
        shape = (128, 128)
        out.append([-rng.uniform(lo, hi, shape), signs(rng, shape) * u * rng.uniform(0.3, 1.1, shape),
                    signs(rng, shape) * dh * rng.uniform(0.3, 1.1, shape)])
    return [oracle.bf16_rne(np.concatenate(t, 1).astype(np.float32)) for t in zip(*out)]


@MODES
def test_gated_far_from_zero(mode):
    g, u, dh = tiles(1)
    I = g.shape[1]
    gu = dev_bf16(np.concatenate([g, u], 1))
    q, s, qc, sc = fb.fp8_gated_forward(gu, scale_mode=mode)
    got = expect(q, s, *unit(f64(g), f64(u)), mode)
    assert (np.abs(got).max(1) > 0).all()
    # (under the power-of-two rule no rounding: a code of the largest u stands for 2^128)
    kept = train_ref.dequant(host(qc), host(sc)) if mode == POW2 else f64(train_ref.kept(host(qc), host(sc)))
    gk, uk, d = kept[:, :I], kept[:, I:], f64(dh)
    assert mode == FP32 or (np.abs(uk) == 2.0 ** 128).any()
    q, s, qT, sT, qhT, shT = fb.fp8_gated_backward(dev_bf16(dh), qc, sc, scale_mode=mode)
    (dg, edg), (du, edu) = gradient(gk, uk, d)
    grad, err = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)
    got = expect(q, s, grad, err, mode)
    assert (np.abs(got[:, :I]).reshape(128, -1, 128).max(2) > 0).all()
    expect(qT, sT, np.ascontiguousarray(grad.T), np.ascontiguousarray(err.T), mode)
    h, eh = unit(gk, uk)
    expect(qhT, shT, np.ascontiguousarray(h.T), np.ascontiguousarray(eh.T), mode)


@pytest.mark.parametrize("value", [2.0 ** 128, -2.0 ** 128])
def test_codes_that_stand_for_two_to_the_128(value):
    """The largest bf16 values are rounded up to it by the power-of-two rule; beside it the unit is an ordinary one for
    some g or u, dh of 0 among them."""
    rng = synth.rng_for(904)
    I, top = 256, np.sign(value) * 3.3895e38
    g, u = rng.uniform(-30, -1, (128, I)), signs(rng, (128, I))
    g[:, ::3], u[:, 1::3] = top if value < 0 else 1e3, top
    g[:, 2::3] = -3.3e38 if value < 0 else -5.0
    dh = rng.uniform(0.5, 1.0, (128, I)) * 1e-3
    dh[:, ::7] = 0.0
    gu, dh = (oracle.bf16_rne(v.astype(np.float32)) for v in (np.concatenate([g, u], 1), dh))
    _, _, qc, sc = fb.fp8_gated_forward(dev_bf16(gu))
    kept = train_ref.dequant(host(qc), host(sc))
    assert (kept == value).any()
    gk, uk, d = kept[:, :I], kept[:, I:], f64(dh)
    with np.errstate(over="ignore"):
        (dg, edg), (du, edu) = gradient(gk, uk, d)
    q, s, _, _, _, _ = fb.fp8_gated_backward(dev_bf16(dh), qc, sc)
    expect(q, s, np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1), POW2)


@MODES
def test_gated_every_g(mode):
    """Each bf16 g from -1 down to -400 for itself: a row of it, times u of one size."""
    g = f64(np.arange(0xBF80, 0xC3C8, dtype=np.uint16))
    u = np.where(g < -80, 3e38, 1e30)
    g, u = (np.repeat(v[:, None], 128, 1) for v in (g, u))
    bits = oracle.bf16_rne(np.concatenate([g, u], 1).astype(np.float32))
    q, s = fb.fp8_gated_forward(dev_bf16(bits), checkpoint=False, scale_mode=mode)
    h, err = unit(g, f64(bits[:, 128:]))
    expect(q, s, h, err, mode)


@MODES
def test_values_beside_those_far_from_zero_are_the_same(mode):
    """Rows of ordinary values in tiles (and waves) that hold others."""
    M, I = 256, 256
    gu, dh = synth.normal_bf16((M, 2 * I), 2.0, 902), synth.normal_bf16((M, I), 1e-2, 903)
    mixed, dmixed = gu.copy(), dh.copy()
    far = np.arange(M) % 5 == 2
    g, u, d = tiles(2)
    mixed[far, :I], mixed[far, I:], dmixed[far] = g[:far.sum(), :I], u[:far.sum(), :I], d[:far.sum(), :I]
    plain = fb.fp8_gated_forward(dev_bf16(gu), scale_mode=mode)
    got = fb.fp8_gated_forward(dev_bf16(mixed), scale_mode=mode)
    for a, b in zip(got, plain):
        assert np.array_equal(host(a)[~far], host(b)[~far])
    plain = fb.fp8_gated_backward(dev_bf16(dh), *plain[2:], scale_mode=mode)
    got = fb.fp8_gated_backward(dev_bf16(dmixed), *got[2:], scale_mode=mode)
    for a, b in zip(got[:2], plain[:2]):
        assert np.array_equal(host(a)[~far], host(b)[~far])


# ------------------------------------------------------------- the quotient --

def test_quotients_at_the_ends_of_the_range():
    """amax / 448 where the short quotient ends and another takes over, and up to the largest amax: every mantissa of the
    amax, elements of 12 octaves below it."""
    rng = synth.rng_for(905)
    top = np.concatenate([np.arange(e << 7, (e + 1) << 7) for e in (*range(127 - 58, 127 - 52), *range(127 + 106, 255))])
    top = np.repeat(top, 4)
    x = np.maximum(top[:, None] - rng.integers(0, 12 * 128, (top.size, 128)), 0)
    x[:, 5] = top
    x = (x | (rng.integers(0, 2, x.shape) << 15)).astype(np.uint16)
    n = len(x)
    assert n % 128 == 0
    source = dev(np.arange(n, dtype=np.int32))
    want = oracle.quantize_rowgroup(x, mode=FP32)
    for got in (fb.fp8_moe_gather(dev_bf16(x), source, 1, scale_mode=FP32),
                fb.fp8_moe_gather(dev_bf16(x), source, 1, transpose=True, scale_mode=FP32)[:2],
                fb.fp8_gated_forward(dev_bf16(np.concatenate([x, x], 1)), scale_mode=FP32)[2:]):
        k = got[1].shape[1]
        assert np.array_equal(host(got[0]), np.tile(want[0], (1, k))) and np.array_equal(host(got[1]), np.tile(want[1], (1, k)))
    across = np.ascontiguousarray(x.T)
    qT, sT = fb.fp8_moe_gather(dev_bf16(across), source[:128].contiguous(), 1, transpose=True, scale_mode=FP32)[2:]
    assert np.array_equal(host(qT), want[0]) and np.array_equal(host(sT), want[1])
