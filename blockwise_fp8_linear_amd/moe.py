"""Binding of include/fp8moe.h: the FP8 linear layer at any number of tokens,
the router of a mixture of experts with its gradient, and a whole
mixture-of-experts layer for a few tokens.

The manner is the package's: the C entry points' names, torch tensors on the
current device, checks of dtype, layout and shape before any C call,
RuntimeError on a non-zero status.  The calls record nothing for autograd,
whatever `requires_grad` says, and return tensors without a gradient:
fp8_moe_route_backward and the package's Dgrad and Wgrad are called by the
user's own autograd function.  These calls stand in decoding loops, where
their own cost is what a caller waits for, so the checks of an operand are one
function and the stream is taken as a raw handle.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

import blockwise_fp8_linear_amd as _fb

HEADER_PATH = os.path.join(os.path.dirname(_fb.HEADER_PATH), "fp8moe.h")

# enum values and limits of include/fp8moe.h
FP8_LINEAR_FP32_ROWS = 127
FP8MOE_BF16 = 0
FP8MOE_FP32 = 1
FP8MOE_MAX_EXPERTS = 1024
FP8MOE_MAX_TOPK = 16
FP8MOE_MAX_TOKENS = 512

_FUNCTIONS = None
_REFUSED = ctypes.c_size_t(-1).value


def _functions():
    """The entry points with their signatures set (once per loaded library)."""
    global _FUNCTIONS
    lib = _fb.load_library()
    if _FUNCTIONS is not None and _FUNCTIONS[0] is lib:
        return _FUNCTIONS[1]
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "fp8_linear": [i64, i64, i64, vp, i64, vp, vp, vp, i32, i32, vp, sz, vp],
        "fp8_moe_route": [i64, i64, i32, vp, i32, i64, i32, vp, vp, vp],
        "fp8_moe_route_backward": [i64, i64, i32, vp, i32, i64, vp, vp, i32, vp, i64, vp],
        "fp8_moe_experts": [i64, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, sz, vp],
        "fp8_moe_layer": [i64, i64, i64, i64, i32, i32, vp, i64, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, sz,
                          vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, i32
    lib.fp8_linear_workspace_size.argtypes = [i64, i64, i64, i32]
    lib.fp8_linear_workspace_size.restype = sz
    lib.fp8_moe_workspace_size.argtypes = [i64, i64, i64, i64, i32]
    lib.fp8_moe_workspace_size.restype = sz
    _FUNCTIONS = (lib, lib)
    return lib


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# torch's own raw-handle query where it has one: the public one builds a Stream
# object, 2 us a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _stream(stream, index):
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _index(x, name):
    """The device a call runs on, by number: its first operand's, which has to
    be the current one (the library launches there)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    index = x.get_device()
    if index < 0:
        raise ValueError(f"{name}: must be a device tensor")
    if index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {x.device}, but the library launches on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    return index


def _new(like, shape, dtype, stream):
    """A new tensor on `like`'s device whose memory belongs to the stream the
    call launches on."""
    if stream is not None:
        return _fb._new(shape, dtype, like.device, stream)
    # dense; the strided form of torch.empty takes the least time of them
    return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=like.device)


def _operand(t, dtype, shape, name, index, strided=False):
    """Check one tensor: on this device, of this dtype and shape, dense (or,
    `strided`, with a contiguous last dimension).  Returns its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, but the call runs on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if strided:
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
    elif not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _matrix(x, dtypes, name):
    """The first operand: a matrix of one of these types, rows any distance
    apart.  Returns its device, sizes and row stride (a single row has none
    that matters)."""
    index = _index(x, name)
    if x.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"{name}: expected 2 dims, got {x.dim()}")
    rows, cols = x.shape
    down, right = x.stride()
    if right != 1 and cols > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return index, rows, cols, down if rows > 1 else cols


def _result(out, like, shape, dtype, name, index, stream):
    """(the output, new or the caller's, and its address)."""
    if out is None:
        out = _new(like, shape, dtype, stream)
        return out, out.data_ptr()
    return out, _operand(out, dtype, shape, name, index)


def _scratch(need, workspace, like, index, stream):
    """(the workspace, to be kept until the call has been made, its address and
    size); nothing where the shape needs none or is refused."""
    if need == 0 or _invalid(need):
        return None, None, 0
    if workspace is None:
        # belongs to `stream`: freed when the call returns, its memory is
        # reused only by work queued behind the kernels that use it
        workspace = _new(like, (need,), torch.uint8, stream)
        return workspace, workspace.data_ptr(), need
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if workspace.get_device() != index:
        raise ValueError(f"workspace: on {workspace.device}, but the call runs on cuda:{index}")
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _topk(k, E):
    """Refuse what a C int would not hold.  Returns whether the call will take k
    choices of E: if not, it says why, and no output is made for it."""
    if not -2**31 <= k < 2**31:
        raise ValueError(f"topk: {k} is not between 1 and {FP8MOE_MAX_TOPK}")
    return 1 <= k <= min(E, FP8MOE_MAX_TOPK)


@functools.lru_cache(maxsize=4096)
def _linear_need(M, N, K, scale_mode):
    return _functions().fp8_linear_workspace_size(M, N, K, scale_mode)


@functools.lru_cache(maxsize=4096)
def _moe_need(T, H, I, E, k):
    return _functions().fp8_moe_workspace_size(T, H, I, E, k)


def _invalid(need):
    """Whether a workspace query refused the shape (the call then says why)."""
    return need == _REFUSED


# ------------------------------------------------------------------- linear --

def fp8_linear_workspace_size(M: int, N: int, K: int, scale_mode: int = _fb.FP8BLK_SCALE_POW2) -> int:
    return int(_functions().fp8_linear_workspace_size(M, N, K, scale_mode))


def fp8_linear(x, qw, sw, out_dtype=None, out=None, workspace=None, stream=None, accumulate=False,
               scale_mode=_fb.FP8BLK_SCALE_POW2):
    """Y = X W^T for any number of tokens.  x bf16 [M,K] (row stride may exceed
    K), qw [N,K] and sw [N/128,K/128] from fp8_quantize_block -> Y [M,N] bf16
    or fp32.  x is quantized on the way by scale_mode's rule, the one that made
    sw.  accumulate: out += result in fp32 (out_dtype float32, `out` given)."""
    bf16 = torch.bfloat16
    index, M, K, ld = _matrix(x, (bf16,), "x")
    if not isinstance(qw, torch.Tensor) or qw.dim() != 2:
        raise ValueError("qw: expected a 2-dim tensor")
    N = qw.shape[0]
    pqw = _operand(qw, torch.uint8, (N, K), "qw", index)
    psw = _operand(sw, torch.float32, (N // 128, K // 128), "sw", index)
    odt = _fb.FP8BLK_OUT_BF16
    if out_dtype is None:
        out_dtype = bf16
    if accumulate or out_dtype is not bf16:
        odt = _fb._odt(out_dtype, accumulate, out)
    lib = _functions()
    keep, ws, size = _scratch(_linear_need(M, N, K, scale_mode), workspace, x, index, stream)
    y, py = _result(out, x, (M, N), out_dtype, "out", index, stream)
    rc = lib.fp8_linear(M, N, K, x.data_ptr(), ld, pqw, psw, py, odt, scale_mode, ws, size, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return y


# ------------------------------------------------------------------- router --

_LOGITS = (torch.bfloat16, torch.float32)


def fp8_moe_route(logits, topk, renormalize=True, ids=None, weights=None, stream=None):
    """The router's choice.  logits bf16 or fp32 [T,E] (row stride may exceed
    E) -> (ids int32 [T,topk], weights fp32 [T,topk]): each token's experts with
    the largest logits, largest first, equal ones by lower index, and their
    softmax weights -- over the chosen ones (renormalize) or over all.  Experts
    whose logit is -inf or NaN are masked out; where fewer than topk are left
    the rest of the row is id -1, weight 0.  Nothing is recorded for autograd:
    fp8_moe_route_backward gives the gradient."""
    index, T, E, ld = _matrix(logits, _LOGITS, "logits")
    pids = pw = None
    if _topk(topk, E):
        ids, pids = _result(ids, logits, (T, topk), torch.int32, "ids", index, stream)
        weights, pw = _result(weights, logits, (T, topk), torch.float32, "weights", index, stream)
    rc = _functions().fp8_moe_route(T, E, topk, logits.data_ptr(),
                                    FP8MOE_FP32 if logits.dtype is torch.float32 else FP8MOE_BF16, ld,
                                    1 if renormalize else 0, pids, pw, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return ids, weights


def fp8_moe_route_backward(logits, ids, dweights, renormalize=True, dlogits=None, stream=None):
    """Gradient of fp8_moe_route's weights: logits and ids as it took and gave
    them, dweights fp32 [T,topk] -> dlogits [T,E] in the logits' type (or into
    `dlogits`, whose row stride may exceed E)."""
    index, T, E, ld = _matrix(logits, _LOGITS, "logits")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids: expected a 2-dim tensor")
    k = ids.shape[1]
    _topk(k, E)
    pids = _operand(ids, torch.int32, (T, k), "ids", index)
    pg = _operand(dweights, torch.float32, (T, k), "dweights", index)
    dtype = logits.dtype
    if dlogits is None:
        dlogits, ld_d = _new(logits, (T, E), dtype, stream), E
    else:
        _operand(dlogits, dtype, (T, E), "dlogits", index, strided=True)
        ld_d = dlogits.stride(0) if T > 1 else E
    rc = _functions().fp8_moe_route_backward(T, E, k, logits.data_ptr(),
                                             FP8MOE_FP32 if dtype is torch.float32 else FP8MOE_BF16, ld, pids, pg,
                                             1 if renormalize else 0, dlogits.data_ptr(), ld_d,
                                             _stream(stream, index))
    if rc:
        _fb._check(rc)
    return dlogits


# ------------------------------------------------------------------ experts --

def fp8_moe_workspace_size(T: int, H: int, I: int, E: int, topk: int) -> int:
    return int(_functions().fp8_moe_workspace_size(T, H, I, E, topk))


def _experts(qw1, sw1, qw2, sw2, H, index):
    """(E, I, the four addresses) of the experts' weights for a hidden size H."""
    if not isinstance(qw1, torch.Tensor) or qw1.dim() != 3 or qw1.shape[1] % 2:
        raise ValueError("qw1: expected a 3-dim tensor [E, 2 I, H]")
    E, I = qw1.shape[0], qw1.shape[1] // 2
    return (E, I, _operand(qw1, torch.uint8, (E, 2 * I, H), "qw1", index),
            _operand(sw1, torch.float32, (E, 2 * I // 128, H // 128), "sw1", index),
            _operand(qw2, torch.uint8, (E, H, I), "qw2", index),
            _operand(sw2, torch.float32, (E, H // 128, I // 128), "sw2", index))


def fp8_moe_experts(x, ids, weights, qw1, sw1, qw2, sw2, out_dtype=None, out=None, workspace=None, stream=None,
                    scale_mode=_fb.FP8BLK_SCALE_POW2):
    """The experts of a mixture for a few tokens (at most FP8MOE_MAX_TOKENS):
    y[t] = sum_i weights[t,i] Wd[e] (silu(G[e] x[t]) * (U[e] x[t])), e =
    ids[t,i]; ids that are no expert (-1) are left out.  x bf16 [T,H] (row
    stride may exceed H); ids int32, weights fp32 [T,topk]; qw1 [E,2I,H] (G's
    rows, then U's) and qw2 [E,H,I] codes, sw1 [E,2I/128,H/128] and sw2
    [E,H/128,I/128], each as fp8_quantize_block quantizes the stacked matrix
    -> y [T,H] bf16 or fp32.  Activations are quantized by scale_mode's rule,
    the one that made the weights' scales."""
    index, T, H, ld = _matrix(x, (torch.bfloat16,), "x")
    E, I, pq1, ps1, pq2, ps2 = _experts(qw1, sw1, qw2, sw2, H, index)
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids: expected a 2-dim tensor")
    k = ids.shape[1]
    pids = _operand(ids, torch.int32, (T, k), "ids", index)
    pw = _operand(weights, torch.float32, (T, k), "weights", index)
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    odt = _fb._odt(out_dtype)
    _topk(k, E)
    lib = _functions()
    keep, ws, size = _scratch(_moe_need(T, H, I, E, k), workspace, x, index, stream)
    y, py = _result(out, x, (T, H), out_dtype, "out", index, stream)
    rc = lib.fp8_moe_experts(T, H, I, E, k, x.data_ptr(), ld, pids, pw, pq1, ps1, pq2, ps2, py, odt, scale_mode, ws,
                             size, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return y


def fp8_moe_layer(x, wr, qw1, sw1, qw2, sw2, topk, renormalize=True, out_dtype=None, out=None, ids=None,
                  weights=None, workspace=None, stream=None, scale_mode=_fb.FP8BLK_SCALE_POW2):
    """A whole mixture-of-experts layer for a few tokens: router logits x wr^T
    (wr bf16 [E,H]), fp8_moe_route's choice of topk experts, fp8_moe_experts of
    it.  `ids` (int32) and `weights` (fp32) [T,topk], where given, get the
    choice.  A token whose logits are all NaN or -inf (its row of x, wr or their
    product is not finite) gets ids -1, weights 0 and a row of NaN."""
    index, T, H, ld = _matrix(x, (torch.bfloat16,), "x")
    E, I, pq1, ps1, pq2, ps2 = _experts(qw1, sw1, qw2, sw2, H, index)
    pwr = _operand(wr, torch.bfloat16, (E, H), "wr", index)
    pids = None if ids is None else _operand(ids, torch.int32, (T, topk), "ids", index)
    pw = None if weights is None else _operand(weights, torch.float32, (T, topk), "weights", index)
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    odt = _fb._odt(out_dtype)
    _topk(topk, E)
    lib = _functions()
    keep, ws, size = _scratch(_moe_need(T, H, I, E, topk), workspace, x, index, stream)
    y, py = _result(out, x, (T, H), out_dtype, "out", index, stream)
    rc = lib.fp8_moe_layer(T, H, I, E, topk, 1 if renormalize else 0, x.data_ptr(), ld, pwr, pq1, ps1, pq2, ps2, py,
                           odt, scale_mode, pids, pw, ws, size, _stream(stream, index))
    if rc:
        _fb._check(rc)
    return y
