"""Binding of include/fp8train.h: training a mixture of experts on the FP8
linear layer -- tokens sorted by expert and back, every expert's products over
its own rows, their gradients -- and what the backward pass needs kept in 8 bits.

The manner is that of moe.py: the C entry points' names, torch tensors on the
current device, checks of dtype, layout and shape before any C call,
RuntimeError on a non-zero status, nothing recorded for autograd.  Outputs may
be given, as a training loop keeps them; those that are not are new, and hold
whatever the memory held in the rows behind the last segment, which no call
writes.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

import blockwise_fp8_linear_amd as _fb

from .moe import _index, _invalid, _matrix, _operand, _raw_stream, _result, _scratch, _topk

HEADER_PATH = os.path.join(os.path.dirname(_fb.HEADER_PATH), "fp8train.h")

_FUNCTIONS = None
_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _functions():
    """The entry points with their signatures set (once per loaded library)."""
    global _FUNCTIONS
    lib = _fb.load_library()
    if _FUNCTIONS is lib:
        return lib
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    gemm = [i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, i32, i32, vp]
    sig = {
        "fp8_moe_sort": [i64, i64, i32, vp, vp, vp, vp, vp, sz, vp],
        "fp8_moe_gather": [i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, i64, vp, vp, i64, vp, i32, vp, sz, vp],
        "fp8_moe_combine": [i64, i64, i64, i32, vp, i64, vp, vp, vp, i32, vp],
        "fp8_moe_combine_backward": [i64, i64, i64, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, vp, i64, vp, vp,
                                     i32, vp],
        "fp8_moe_gemm_fprop": gemm,
        "fp8_moe_gemm_dgrad": gemm,
        "fp8_moe_gemm_wgrad": gemm,
        "fp8_gated_forward": [i64, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, i32, vp],
        "fp8_gated_backward": [i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, i64, vp, vp, i64, vp, i32, vp],
        "fp8_requantize_colgroup": [vp, i64, i64, i64, vp, vp, vp, i64, vp, i32, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, i32
    for name in ("fp8_moe_sorted_rows", "fp8_moe_sort_workspace_size"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [i64, i64, i32], sz
    lib.fp8_moe_gather_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    lib.fp8_moe_gather_workspace_size.restype = sz
    _FUNCTIONS = lib
    return lib


def _stream(stream, index):
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _codes(q, s, rows, cols, name, like, index, stream, groups=None):
    """Outputs of a quantizer, new or the caller's: (q, its address, its row
    stride, s, its address).  Scales are dense, codes may have a wider row."""
    if q is None:
        q = _new(like, (rows, cols), _U8, stream)
        pq, ld = q.data_ptr(), cols
    else:
        pq = _operand(q, _U8, (rows, cols), name, index, strided=True)
        ld = q.stride(0) if rows > 1 else cols
    s, ps = _result(s, like, (rows, cols // 128), _F32, "scales of " + name, index, stream)
    return q, pq, ld, s, ps


def _new(like, shape, dtype, stream):
    if stream is not None:
        return _fb._new(shape, dtype, like.device, stream)
    return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=like.device)


def _kept(q, s, name):
    """Row-group codes as a first operand: (device, rows, cols, row stride, the
    address of the scales)."""
    index, rows, cols, ld = _matrix(q, (_U8,), name)
    return index, rows, cols, ld, _operand(s, _F32, (rows, cols // 128), "scales of " + name, index)


def _limit(used, index):
    return None if used is None else _operand(used, _I32, (1,), "used", index)


def _choices(t, dtype, name, index):
    """A [T, k] operand: (k, its address)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-dim tensor")
    return t.shape[1], _operand(t, dtype, tuple(t.shape), name, index)


# ---------------------------------------------------------- sorted by expert --

@functools.lru_cache(maxsize=4096)
def _sort_sizes(T, E, k):
    lib = _functions()
    return lib.fp8_moe_sorted_rows(T, E, k), lib.fp8_moe_sort_workspace_size(T, E, k)


def _size(n, what, T, E, topk):
    if _invalid(n):
        raise ValueError(f"{what}: no such choice: T {T}, E {E}, topk {topk}")
    return int(n)


def fp8_moe_sorted_rows(T: int, E: int, topk: int) -> int:
    """Rows that any choice of topk of E experts by T tokens fits in."""
    return _size(_sort_sizes(T, E, topk)[0], "fp8_moe_sorted_rows", T, E, topk)


def fp8_moe_sort_workspace_size(T: int, E: int, topk: int) -> int:
    return _size(_sort_sizes(T, E, topk)[1], "fp8_moe_sort_workspace_size", T, E, topk)


def fp8_moe_sort(ids, E, rows=None, source=None, offsets=None, workspace=None, stream=None):
    """The sorted order of a choice.  ids int32 [T,k] -> (rows int32 [T,k], the
    sorted row of each choice, -1 where the id is no expert; source int32 [R],
    the choice t k + i of each row, -1 for padding; offsets int32 [E+1], the
    segments' first rows, multiples of 128).  R = fp8_moe_sorted_rows(T, E, k);
    offsets[-1:] is the `used` of the calls below."""
    index = _index(ids, "ids")
    k, pids = _choices(ids, _I32, "ids", index)
    T = ids.shape[0]
    lib = _functions()
    R, need = _sort_sizes(T, E, k)
    pr = ps = po = None
    if not _invalid(R):
        rows, pr = _result(rows, ids, (T, k), _I32, "rows", index, stream)
        source, ps = _result(source, ids, (R,), _I32, "source", index, stream)
        offsets, po = _result(offsets, ids, (E + 1,), _I32, "offsets", index, stream)
    else:
        pr = ps = po = pids  # refused before any of them is looked at
    keep, ws, size = _scratch(need, workspace, ids, index, stream)
    rc = lib.fp8_moe_sort(T, E, k, pids, pr, ps, po, ws, size, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return rows, source, offsets


@functools.lru_cache(maxsize=4096)
def _gather_need(T, H, R, k, transpose):
    return _functions().fp8_moe_gather_workspace_size(T, H, R, k, transpose)


def fp8_moe_gather_workspace_size(T: int, H: int, R: int, topk: int, transpose: bool = False) -> int:
    need = _gather_need(T, H, R, topk, 1 if transpose else 0)
    if _invalid(need):
        raise ValueError(f"fp8_moe_gather_workspace_size: no such gather: T {T}, H {H}, R {R}, topk {topk}")
    return int(need)


def fp8_moe_gather(x, source, topk, used=None, weights=None, transpose=False, q=None, s=None, qT=None, sT=None,
                   workspace=None, stream=None, scale_mode=_fb.FP8BLK_SCALE_POW2):
    """The tokens' rows in sorted order, quantized.  x bf16 [T,H] (row stride may
    exceed H), source int32 [R] -> (q uint8 [R,H], s fp32 [R,H/128]), or with
    transpose (q, s, qT uint8 [H,R], sT fp32 [H,R/128]): the codes that
    fp8_quantize_rowgroup (and _colgroup) give for the rows x[source[r] // topk],
    or bf16(weights.view(-1)[source[r]] * that) where weights fp32 [T,topk] are
    given; zeros where source is no choice.  used: int32 [1] on the device, the
    rows to do (None: all)."""
    index, T, H, ld = _matrix(x, (_BF16,), "x")
    if not isinstance(source, torch.Tensor) or source.dim() != 1:
        raise ValueError("source: expected a 1-dim tensor")
    R = source.shape[0]
    psource = _operand(source, _I32, (R,), "source", index)
    _topk(topk, topk)
    pw = None if weights is None else _operand(weights, _F32, (T, topk), "weights", index)
    pused = _limit(used, index)
    q, pq, ldq, s, ps = _codes(q, s, R, H, "q", x, index, stream)
    pqT, ldT, psT = None, 0, None
    if transpose:
        qT, pqT, ldT, sT, psT = _codes(qT, sT, H, R, "qT", x, index, stream)
    lib = _functions()
    keep, ws, size = _scratch(_gather_need(T, H, R, topk, 1 if transpose else 0), workspace, x, index, stream)
    rc = lib.fp8_moe_gather(T, H, R, topk, x.data_ptr(), ld, psource, pw, pused, pq, ldq, ps, pqT, ldT, psT, scale_mode,
                            ws, size, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return (q, s, qT, sT) if transpose else (q, s)


def fp8_moe_combine(z, rows, weights=None, out_dtype=None, out=None, stream=None, accumulate=False):
    """Sorted rows back to their tokens: y[t] = sum_i weights[t,i] z[rows[t,i]],
    rows that are -1 left out.  z bf16 [R,H] (row stride may exceed H), rows int32
    [T,k], weights fp32 [T,k] or None for 1 (the gradient of fp8_moe_gather) -> y
    [T,H] bf16 or fp32.  accumulate: out += result (out_dtype float32, `out`
    given)."""
    index, R, H, ld = _matrix(z, (_BF16,), "z")
    k, prows = _choices(rows, _I32, "rows", index)
    T = rows.shape[0]
    pw = None if weights is None else _operand(weights, _F32, (T, k), "weights", index)
    out_dtype = _BF16 if out_dtype is None else out_dtype
    odt = _fb._odt(out_dtype, accumulate, out)
    y, py = _result(out, z, (T, H), out_dtype, "out", index, stream)
    rc = _functions().fp8_moe_combine(T, H, R, k, z.data_ptr(), ld, prows, pw, py, odt, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return y


def fp8_moe_combine_backward(dy, z, rows, source, weights, used=None, q=None, s=None, qT=None, sT=None, dweights=None,
                             stream=None, scale_mode=_fb.FP8BLK_SCALE_POW2):
    """Gradient of fp8_moe_combine with weights.  dy bf16 [T,H]; z, rows, weights
    as it took them; source int32 [R] -> (q [R,H], s, qT [H,R], sT, dweights fp32
    [T,k]): the gradients of the rows, weights[t,i] dy[t] rounded to bf16, in both
    orientations, and of the weights, <dy[t], z[rows[t,i]]>."""
    index, T, H, ld = _matrix(dy, (_BF16,), "dy")
    _, R, _, ld_z = _matrix(z, (_BF16,), "z")
    pz = _operand(z, _BF16, (R, H), "z", index, strided=True)
    if not isinstance(rows, torch.Tensor) or rows.dim() != 2:
        raise ValueError("rows: expected a 2-dim tensor")
    k = rows.shape[1]
    prows = _operand(rows, _I32, (T, k), "rows", index)
    psource = _operand(source, _I32, (R,), "source", index)
    pw = _operand(weights, _F32, (T, k), "weights", index)
    pused = _limit(used, index)
    q, pq, ldq, s, ps = _codes(q, s, R, H, "q", dy, index, stream)
    qT, pqT, ldT, sT, psT = _codes(qT, sT, H, R, "qT", dy, index, stream)
    dweights, pd = _result(dweights, dy, (T, k), _F32, "dweights", index, stream)
    rc = _functions().fp8_moe_combine_backward(T, H, R, k, dy.data_ptr(), ld, pz, ld_z, prows, psource, pw, pused, pq,
                                               ldq, ps, pqT, ldT, psT, pd, scale_mode, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return q, s, qT, sT, dweights


# ------------------------------------------------------- the experts' products --

def _gemm(name, sizes, a, sa, b, sb, offsets, shape, out_dtype, out, stream, accumulate, scale_mode, index):
    R, N, K, E = sizes
    poff = _operand(offsets, _I32, (E + 1,), "offsets", index)
    out_dtype = _BF16 if out_dtype is None else out_dtype
    odt = _fb._odt(out_dtype, accumulate, out)
    if out is None:
        out = _fb._new(shape, out_dtype, a.device, stream)
        py = out.data_ptr()
    else:
        py = _operand(out, out_dtype, shape, "out", index)
    rc = getattr(_functions(), name)(R, N, K, E, a.data_ptr(), sa, b.data_ptr(), sb, poff, py, odt, scale_mode,
                                     _stream(stream, index))
    if rc:
        _fb._check(rc)
    return out


def _weights(qw, sw, index):
    """Sizes (E, N, K) of the experts' weights and the address of their scales."""
    if not isinstance(qw, torch.Tensor) or qw.dim() != 3:
        raise ValueError("qw: expected a 3-dim tensor [E, N, K]")
    E, N, K = qw.shape
    _operand(qw, _U8, (E, N, K), "qw", index)
    return E, N, K, _operand(sw, _F32, (E, N // 128, K // 128), "sw", index)


def fp8_moe_gemm_fprop(qx, sx, qw, sw, offsets, out_dtype=None, out=None, stream=None, accumulate=False,
                       scale_mode=_fb.FP8BLK_SCALE_POW2):
    """y[r] = x[r] W_e^T for the rows r of expert e's segment [offsets[e],
    offsets[e+1]).  qx [R,K] + sx [R,K/128], qw [E,N,K] + sw [E,N/128,K/128],
    offsets int32 [E+1] -> y [R,N] bf16 or fp32; rows of no segment are not
    written.  accumulate: out += result in fp32."""
    index = _index(qx, "qx")
    E, N, K, psw = _weights(qw, sw, index)
    R = qx.shape[0]
    _operand(qx, _U8, (R, K), "qx", index)
    psx = _operand(sx, _F32, (R, K // 128), "sx", index)
    return _gemm("fp8_moe_gemm_fprop", (R, N, K, E), qx, psx, qw, psw, offsets, (R, N), out_dtype, out, stream,
                 accumulate, scale_mode, index)


def fp8_moe_gemm_dgrad(qdy, sdy, qw, sw, offsets, out_dtype=None, out=None, stream=None, accumulate=False,
                       scale_mode=_fb.FP8BLK_SCALE_POW2):
    """dx[r] = dy[r] W_e from the weight codes as quantized.  qdy [R,N] + sdy
    [R,N/128], qw [E,N,K] + sw -> dx [R,K]; the rest as fp8_moe_gemm_fprop."""
    index = _index(qdy, "qdy")
    E, N, K, psw = _weights(qw, sw, index)
    R = qdy.shape[0]
    _operand(qdy, _U8, (R, N), "qdy", index)
    psd = _operand(sdy, _F32, (R, N // 128), "sdy", index)
    return _gemm("fp8_moe_gemm_dgrad", (R, N, K, E), qdy, psd, qw, psw, offsets, (R, K), out_dtype, out, stream,
                 accumulate, scale_mode, index)


def fp8_moe_gemm_wgrad(qdyT, sdyT, qxT, sxT, offsets, out_dtype=None, out=None, stream=None, accumulate=False,
                       scale_mode=_fb.FP8BLK_SCALE_POW2):
    """dW_e = sum over expert e's rows of dy^T x.  qdyT [N,R] + sdyT [N,R/128],
    qxT [K,R] + sxT [K,R/128], offsets int32 [E+1] -> dw [E,N,K] bf16 or fp32;
    zeros for an expert without rows.  accumulate: out += result in fp32."""
    index = _index(qdyT, "qdyT")
    if qdyT.dim() != 2 or not isinstance(qxT, torch.Tensor) or qxT.dim() != 2:
        raise ValueError("qdyT, qxT: expected 2-dim tensors")
    (N, R), K = qdyT.shape, qxT.shape[0]
    _operand(qdyT, _U8, (N, R), "qdyT", index)
    psd = _operand(sdyT, _F32, (N, R // 128), "sdyT", index)
    _operand(qxT, _U8, (K, R), "qxT", index)
    psx = _operand(sxT, _F32, (K, R // 128), "sxT", index)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets: expected a 1-dim tensor of E + 1")
    E = offsets.shape[0] - 1
    return _gemm("fp8_moe_gemm_wgrad", (R, N, K, E), qdyT, psd, qxT, psx, offsets, (E, N, K), out_dtype, out, stream,
                 accumulate, scale_mode, index)


# --------------------------------------------------------- kept in 8 bits --

def fp8_gated_forward(gu, used=None, checkpoint=True, q=None, s=None, qc=None, sc=None, stream=None,
                      scale_mode=_fb.FP8BLK_SCALE_POW2):
    """h = silu(g) u rounded to bf16 and quantized, and its inputs kept in 8 bits.
    gu bf16 [M,2I] (g's columns, then u's; row stride may exceed 2 I) -> (q uint8
    [M,I], s fp32 [M,I/128], qc uint8 [M,2I], sc fp32 [M,2I/128]); without
    checkpoint (q, s).  used: int32 [1] on the device, the rows to do (None: all)."""
    index, M, cols, ld = _matrix(gu, (_BF16,), "gu")
    if cols % 2:
        raise ValueError("gu: expected [M, 2 I]")
    I = cols // 2
    pused = _limit(used, index)
    q, pq, ldq, s, ps = _codes(q, s, M, I, "q", gu, index, stream)
    pqc, ldc, psc = None, 0, None
    if checkpoint:
        qc, pqc, ldc, sc, psc = _codes(qc, sc, M, cols, "qc", gu, index, stream)
    rc = _functions().fp8_gated_forward(M, I, gu.data_ptr(), ld, pused, pq, ldq, ps, pqc, ldc, psc, scale_mode,
                                        _stream(stream, index))
    if rc:
        _fb._check(rc)
    return (q, s, qc, sc) if checkpoint else (q, s)


def fp8_gated_backward(dh, qc, sc, used=None, q=None, s=None, qT=None, sT=None, qhT=None, shT=None, stream=None,
                       scale_mode=_fb.FP8BLK_SCALE_POW2):
    """The gated unit's gradient from its checkpoint.  dh bf16 [M,I] (row stride
    may exceed I), qc and sc as fp8_gated_forward gave them -> (q [M,2I], s, qT
    [2I,M], sT: the gradients of (g, u) in both orientations; qhT [I,M], shT: h of
    the checkpoint, for the second linear's Wgrad)."""
    index, M, I, ld = _matrix(dh, (_BF16,), "dh")
    _, _, _, ldc, psc = _kept(qc, sc, "qc")
    pqc = _operand(qc, _U8, (M, 2 * I), "qc", index, strided=True)
    pused = _limit(used, index)
    q, pq, ldq, s, ps = _codes(q, s, M, 2 * I, "q", dh, index, stream)
    qT, pqT, ldT, sT, psT = _codes(qT, sT, 2 * I, M, "qT", dh, index, stream)
    qhT, pqh, ldh, shT, psh = _codes(qhT, shT, I, M, "qhT", dh, index, stream)
    rc = _functions().fp8_gated_backward(M, I, dh.data_ptr(), ld, pqc, ldc, psc, pused, pq, ldq, ps, pqT, ldT, psT, pqh,
                                         ldh, psh, scale_mode, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return q, s, qT, sT, qhT, shT


def fp8_requantize_colgroup(q, s, used=None, qT=None, sT=None, stream=None, scale_mode=_fb.FP8BLK_SCALE_POW2):
    """Row groups to column groups: q uint8 [rows,cols] (row stride may exceed
    cols), s fp32 [rows,cols/128] -> (qT uint8 [cols,rows], sT fp32
    [cols,rows/128]), what fp8_quantize_colgroup gives for the values that they
    stand for, rounded to bf16."""
    index, rows, cols, ld, ps = _kept(q, s, "q")
    pused = _limit(used, index)
    qT, pqT, ldT, sT, psT = _codes(qT, sT, cols, rows, "qT", q, index, stream)
    rc = _functions().fp8_requantize_colgroup(q.data_ptr(), rows, cols, ld, ps, pused, pqT, ldT, psT, scale_mode,
                                              _stream(stream, index))
    if rc:
        _fb._check(rc)
    return qT, sT
