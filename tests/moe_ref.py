"""64-bit references of the operators of include/fp8moe.h, on the CPU, with
bounds on how far a correct fp32 implementation may be from them.  The E4M3
codes and scales come from the oracle's quantizers (bit-exact by their own
pins); the rest is written from the definitions in the header."""
from __future__ import annotations

import math

import numpy as np

import oracle

# One rounding to fp32 is off by at most 2^-24 of its result; an accumulator
# that truncates instead, by 2^-23.  The matrix instructions are allowed that.
U = 2.0 ** -24


def f64(bits):
    return oracle.bf16_to_f64(bits)


def dequant_rows(bits, mode):
    """bf16 bits [M, K] -> what their row-group codes stand for, float64."""
    q, s = oracle.quantize_rowgroup(np.ascontiguousarray(bits), mode=mode)
    return oracle.e4m3_decode(q) * np.repeat(s.astype(np.float64), 128, axis=1)


def dequant_block(q, s):
    return oracle.e4m3_decode(q) * np.repeat(np.repeat(s.astype(np.float64), 128, axis=-2), 128, axis=-1)


def product(x, w):
    """x [M, K] w [N, K]^T and the error bound of its fp32 evaluation: per
    128-block 128 additions, then the blocks' and up to 16 waves' sums, and
    roundings of the scale product -- each off by 2 U of the sum of
    magnitudes at most."""
    y = x @ w.T
    nkb = x.shape[1] // 128
    return y, (128 + nkb + 16 + 4) * 2 * U * (np.abs(x) @ np.abs(w).T)


def bf16(v):
    return f64(oracle.bf16_rne(v.astype(np.float32)))


def _scale(amax, mode):
    a = amax.astype(np.float64)
    if mode == oracle.SCALE_FP32:
        s = (a.astype(np.float32) / np.float32(448.0)).astype(np.float64)
    else:
        m, e = np.frexp(a)                     # a = m 2^e; a <= 448 2^k  <=>  m <= 0.875 2^(9 + k - e)
        s = np.ldexp(1.0, np.maximum(e - 9 + (m > 0.875), -126))
    return np.where(a == 0, 1.0, s)


def _codes(b, s, mode):
    """Values of b's E4M3 codes under given scales (one per 128 columns)."""
    s = np.repeat(s, 128, axis=1)
    v = b / s
    if mode == oracle.SCALE_FP32:
        v = v.astype(np.float32).astype(np.float64)
    return oracle.e4m3_decode(oracle.e4m3_encode(np.clip(v, -448.0, 448.0))) * s


def quantize_between(h, err, mode):
    """What bf16(h) quantizes to, and how far it may be off where h is known to
    +-err: the largest difference over both ends of each element's interval and
    both ends of its group's amax."""
    ref_b = bf16(h)
    groups = lambda b: np.abs(b).reshape(b.shape[0], -1, 128).max(2)  # noqa: E731
    ref = _codes(ref_b, _scale(groups(ref_b), mode), mode)
    lo, hi = bf16(np.sign(h) * np.maximum(np.abs(h) - err, 0)), bf16(np.sign(h) * (np.abs(h) + err))
    off = np.zeros_like(h)
    for s in (_scale(groups(lo), mode), _scale(groups(hi), mode)):
        for b in (lo, hi):
            off = np.maximum(off, np.abs(_codes(b, s, mode) - ref))
    return ref, off


def experts(x_bits, ids, weights, qw1, sw1, qw2, sw2, mode):
    """fp8_moe_experts in 64 bits: (y, bound)."""
    x = dequant_rows(x_bits, mode)
    T, k = ids.shape
    E, H, I = qw2.shape
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        gu, egu = product(x[t], dequant_block(qw1[e], sw1[e]))
        g, u, eg, eu = gu[:, :I], gu[:, I:], egu[:, :I], egu[:, I:]
        with np.errstate(over="ignore"):
            silu = g / (1.0 + np.exp(-g))
        # silu' <= 1.1; exp, the sum, the quotient and the product round too (exp to 2 ulp = 4 U at most)
        eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 16 * U * np.abs(silu * u)
        h, oh = quantize_between(silu * u, eh, mode)
        wd = dequant_block(qw2[e], sw2[e])
        p, ep = product(h, wd)
        w = weights[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, w * p)
        # off codes enter times |Wd|; the weighted terms are added with one rounding per term and per block
        np.add.at(bound, t, np.abs(w) * (ep * 2 + oh @ np.abs(wd).T + (k + 4) * 2 * U * np.abs(h) @ np.abs(wd).T))
    return y, bound


def route(logits, k, renorm):
    """(ids, weights) of float64 logits [T, E], row by row."""
    T, E = logits.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        row = logits[t]
        left = [j for j in range(E) if row[j] > -math.inf]
        chosen = sorted(left, key=lambda j: (-row[j], j))[:k]
        p = _softmax(row, chosen if renorm else left)
        for i, j in enumerate(chosen):
            ids[t, i], weights[t, i] = j, p[j]
    return ids, weights


def _softmax(row, among):
    top = max((row[j] for j in among), default=0.0)
    e = {j: 1.0 if row[j] == top else math.exp(row[j] - top) for j in among}
    z = math.fsum(e.values())
    return {j: v / z for j, v in e.items()}


def route_backward(logits, ids, g, renorm):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        row = logits[t]
        left = [j for j in range(E) if row[j] > -math.inf]
        at = {}
        for i, j in enumerate(ids[t]):
            if 0 <= j < E and row[j] > -math.inf:
                at[int(j)] = at.get(int(j), 0.0) + g[t, i]
        p = _softmax(row, sorted(at) if renorm else left)
        mean = math.fsum(p[j] * v for j, v in at.items())
        for j, v in p.items():
            out[t, j] = v * (at.get(j, 0.0) - mean)
    return out


def route_tolerance(spread, n):
    """Relative error of a softmax weight in fp32: the difference to the top
    (|d| U), exp (2 ulp), a sum of n positive terms, the quotient."""
    return (2 * spread + 8 + n + 4) * U
