"""64-bit references of the operators of include/fp8train.h, on the CPU, with
bounds on how far a correct fp32 implementation may be from them.  E4M3 codes and
scales come from the oracle's quantizers; the rest is written from the
definitions in the header."""
from __future__ import annotations

import numpy as np

import oracle
from moe_ref import U, bf16, f64, quantize_between  # noqa: F401  (for the tests that import this module)


def sorted_rows(T, E, k):
    """Every choice a row, each expert that can be reached 127 of padding, in whole 512s."""
    return -(-(T * k + 127 * min(E, T * k)) // 512) * 512


def sort(ids, E, R):
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for c, e in enumerate(ids.ravel().tolist()):
        if 0 <= e < E:
            lists[e].append(c)
    rows, source, offsets = np.full(T * k, -1, np.int32), np.full(R, -1, np.int32), [0]
    for e in range(E):
        for j, c in enumerate(lists[e]):
            rows[c] = offsets[-1] + j
            source[offsets[-1] + j] = c
        offsets.append(offsets[-1] + -(-len(lists[e]) // 128) * 128)
    return rows.reshape(T, k), source, np.array(offsets, np.int32)


def gathered(x_bits, source, k, weights=None):
    """The sorted rows' bf16 bits before they are quantized: w x is one fp32 product, rounded to bf16."""
    live = (source >= 0) & (source < x_bits.shape[0] * k)
    out = np.zeros((source.size, x_bits.shape[1]), np.uint16)
    v = x_bits[source[live] // k]
    if weights is not None:
        w = weights.ravel()[source[live]].astype(np.float32)[:, None]
        v = oracle.bf16_rne(f64(v).astype(np.float32) * w)
    out[live] = v
    return out


def combine(z, rows, weights):
    """(y, bound): k products added in fp32, one rounding each (an fma) or two."""
    T, k = rows.shape
    y, size = np.zeros((T, z.shape[1])), np.zeros((T, z.shape[1]))
    for i in range(k):
        t = np.nonzero((rows[:, i] >= 0) & (rows[:, i] < z.shape[0]))[0]
        w = np.ones(t.size) if weights is None else weights[t, i].astype(np.float64)
        y[t] += w[:, None] * z[rows[t, i]]
        size[t] += np.abs(w[:, None] * z[rows[t, i]])
    return y, 2 * k * U * size


def dweights(dy, z, rows):
    """(dw, bound): H products added in fp32, in whatever order."""
    T, k = rows.shape
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for i in range(k):
        t = np.nonzero((rows[:, i] >= 0) & (rows[:, i] < z.shape[0]))[0]
        p = dy[t] * z[rows[t, i]]
        dw[t, i], size[t, i] = p.sum(1), np.abs(p).sum(1)
    return dw, 2 * dy.shape[1] * U * size


def sigmoid(g):
    """(sigmoid, bound of an fp32 evaluation by 1 / (1 + 2^(-g log2 e))): the argument is rounded twice (the constant and
    the product), 2 |g| U of e^-g; the power to 2 ulp (4 U), the sum and the quotient one rounding each.  e^-g enters 1
    + e^-g with at most its own share, and below fp32's normal range (2^-126) the quotient may be flushed."""
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return s, (2 * np.abs(g) + 6) * U * s + 2.0 ** -126


def gated(g, u):
    """(h, bound) before its rounding to bf16: two more roundings."""
    s, es = sigmoid(g)
    return g * s * u, np.abs(g * u) * es + 3 * U * np.abs(g * s * u)


def gated_backward(g, u, dh):
    """((dg, bound), (du, bound)): dg = dh u sig (1 + g (1 - sig)), du = dh g sig."""
    s, es = sigmoid(g)
    f = s * (1.0 + g * (1.0 - s))
    # 1 - sig: off by es and one rounding; times g, plus 1, times sig: one rounding each of at most 1 + |g|
    ef = s * (np.abs(g) * (es + 2 * U) + 3 * U * (1.0 + np.abs(g))) + es * (1.0 + np.abs(g))
    return ((dh * u * f, np.abs(dh * u) * ef + 4 * U * np.abs(dh * u * f)),
            (dh * g * s, np.abs(dh * g) * es + 3 * U * np.abs(dh * g * s)))


def dequant(q, s):
    """Row-group codes -> the values that they stand for."""
    return oracle.e4m3_decode(q) * np.repeat(s.astype(np.float64), 128, axis=1)


def kept(q, s):
    """The same as the backward pass takes them: one fp32 product, rounded to bf16."""
    v = oracle.e4m3_decode(q).astype(np.float32) * np.repeat(s, 128, axis=1)
    return oracle.bf16_rne(v)
