"""The operators that train a mixture of experts on the FP8 linear layer, with
what the backward pass needs kept in 8 bits, as they are measured.

  dispatch    fp8_moe_sort and fp8_moe_gather: tokens sorted by expert, their
              rows quantized (E4M3, groups of 128) as they are gathered.
  combine     fp8_moe_combine and fp8_moe_combine_backward: the experts' rows
              back to their tokens, with weights, and the gradient.
  experts     fp8_moe_gemm_fprop / _dgrad / _wgrad: every expert's product with
              its own segment of the sorted rows.
  gated       fp8_gated_forward and fp8_gated_backward: silu(g) u quantized for
              the next product, (g, u) kept as E4M3, and the gradient from that.
  requantize  fp8_requantize_colgroup: the operand of the weights' gradient from
              the row groups that the forward pass kept.

`run` computes them in elementary torch operations where `own` is false and
by the library's entry points where it is true.  Rounding, on both sides as
the library documents it: to bf16 once where the layer has a bf16 tensor
between two products (silu(g) u, a weighted gradient, a kept value), to E4M3
with one scale per 128 values right after, results to the output type once;
everything else in 32 bits or more.  Codes are returned as the E4M3 values
that they are, beside their scales.  Segments of the sorted rows start at
multiples of 128; the rows behind the last segment stay what the program's
buffers held.
"""
import math

import torch

own = False

DEV = "cuda"
POW2, FP32 = "pow2", "amax448"
LOG2E = 1.4426950408889634


# -------------------------------------------------------------------- cases --

def listed():
    return [
        # a handful of tokens to their experts: pure latency
        dict(name="dispatch 7", op="dispatch", T=7, E=8, k=2, H=2048, ld=2048, padded=0, both=False, scale=POW2),
        # a ragged, padded micro-batch whose x is a column slice, both orientations at once, amax / 448 scales
        dict(name="dispatch 4095 padded", op="dispatch", T=4095, E=60, k=4, H=2048, ld=4096, padded=96, both=True,
             scale=FP32),
        # a whole micro-batch of 4 x 4096 tokens through many small experts
        dict(name="dispatch 16384", op="dispatch", T=16384, E=128, k=8, H=2048, ld=2048, padded=0, both=False,
             scale=POW2),
        # the experts' rows of a small batch back to its tokens, in fp32 for a residual stream
        dict(name="combine 33 fp32", op="combine", T=33, E=8, k=2, H=2048, padded=2, out="fp32", back=False, scale=POW2),
        # a micro-batch's rows back to its tokens while training, with the gradients of rows and weights
        dict(name="combine 16384 back", op="combine", T=16384, E=64, k=8, H=2048, padded=0, out="bf16", back=True,
             scale=POW2),
        # few tokens for eight large experts: the weights weigh more than the rows
        dict(name="experts fprop 300", op="experts", T=300, E=8, k=2, N=4096, K=2048, way="fprop", scale=POW2),
        # the gradient of a micro-batch's gate/up input, unevenly loaded experts
        dict(name="experts dgrad 8192", op="experts", T=8192, E=64, k=8, N=2048, K=2048, way="dgrad", scale=POW2),
        # and of the weights
        dict(name="experts wgrad 8192", op="experts", T=8192, E=64, k=8, N=2048, K=2048, way="wgrad", scale=POW2),
        # the gated unit of an odd small batch of rows, amax / 448 scales
        dict(name="gated 200", op="gated", M=200, I=768, used=200, back=False, scale=FP32),
        # the decoder layer's MLP (6144) on a training step's 8192 tokens, forward and backward
        dict(name="gated 8192 back", op="gated", M=8192, I=6144, used=8192, back=True, scale=POW2),
        # the kept input of a small product, turned for the weights' gradient
        dict(name="requantize 384", op="requantize", M=384, C=2048, used=384, scale=POW2),
        # sorted rows of a large mixture, turned; the buffer is larger than what the batch filled
        dict(name="requantize 69632", op="requantize", M=69632, C=2048, used=65536, scale=FP32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "experts", "experts", "gated", "gated", "requantize"])
    scale = rng.choice([POW2, POW2, FP32])
    if op in ("dispatch", "combine"):
        T, E, H = _log(rng, 1, 16384), _log(rng, 2, 256), 128 * _log(rng, 1, 32)
        k = rng.randint(1, min(8, E))
        while T * k * H > 16384 * 8 * 2048:
            T //= 2
        case = dict(op=op, T=T, E=E, k=k, H=H, padded=rng.choice([0, 0, rng.randint(0, T // 4)]))
        if op == "dispatch":
            return dict(case, ld=H + 8 * rng.choice([0, 0, 1, 33]), both=rng.random() < 0.5, scale=scale)
        return dict(case, out=rng.choice(["bf16", "fp32"]), back=rng.random() < 0.5, scale=scale)
    if op == "experts":
        T, E, N, K = _log(rng, 16, 8192), _log(rng, 2, 64), 128 * _log(rng, 2, 48), 128 * _log(rng, 2, 32)
        k = rng.randint(1, min(8, E))
        while E * N * K > 64 * 2048 * 2048:
            E, k = E // 2, min(k, E // 2)
        while T * k * N * K > 8192 * 8 * 2048 * 2048:
            T //= 2
        return dict(op=op, T=T, E=E, k=k, N=N, K=K, way=rng.choice(["fprop", "dgrad", "wgrad"]), scale=scale)
    if op == "gated":
        back = rng.random() < 0.6
        M, I = _log(rng, 1, 16384), 128 * _log(rng, 1, 48)
        while M * I > 8192 * 6144:
            M //= 2
        if back:
            M = 128 * max(1, M // 128)
        return dict(op=op, M=M, I=I, used=rng.choice([M, M, rng.randint(1, max(1, M // 128)) * 128 if M >= 128 else M]),
                    back=back, scale=scale)
    M, C = 128 * _log(rng, 1, 512), 128 * _log(rng, 1, 48)
    while M * C > 69632 * 2048:
        M = M // 256 * 128
    return dict(op=op, M=M, C=C, used=rng.choice([M, M, 128 * rng.randint(1, M // 128)]), scale=scale)


# ------------------------------------------------- E4M3 and its scale rules --

def _scales(amax, rule):
    """The scale of groups with this fp32 amax: the smallest power of two s >= 2^-126 with amax <= 448 s, or
    amax / 448 rounded to fp32; 1 for a group of zeros."""
    if rule == FP32:
        s = amax / torch.full_like(amax, 448.0)  # divided by a tensor: by a number, torch multiplies with its inverse
    else:
        m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
        e = (e - 9 + (m > 0.875).to(e.dtype)).clamp_min(-126)
        s = ((e + 127) << 23).view(torch.float32)  # 2^e by its bits: torch's ldexp goes by pow, which rounds
    return torch.where(amax == 0, torch.ones_like(s), s)


def _codes(x, rule):
    """x fp32 [rows, n * 128] -> E4M3 values [rows, n * 128] and scales [rows, n]."""
    g = x.unflatten(1, (-1, 128))
    s = _scales(g.abs().amax(2, keepdim=True), rule)
    return (g / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(x.shape), s.squeeze(2)


def _codes_t(x, rule):
    """The same in groups of 128 rows of a column, transposed: [cols, rows] and [cols, rows / 128]."""
    return _codes(x.t().contiguous(), rule)


def _value(q, s):
    """What row-group codes stand for, fp32."""
    return (q.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * s[:, :, None]).flatten(1)


def _decode(q, s):
    """E4M3 codes [..., R, C] with block scales [..., R/128, C/128] -> fp32 values."""
    w = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    return (w * s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)


def _weight(shape, std, rule, gen):
    """A weight ~ N(0, std) in E4M3 blocks: codes (uint8, `shape`) and block scales."""
    w = (torch.randn(shape, generator=gen, device=DEV) * std).bfloat16().float()
    w = w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    s = _scales(w.abs().amax((-1, -3), keepdim=True), rule)
    q = (w / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten(-2).flatten(-3, -2).contiguous(), s.squeeze(-1).squeeze(-2).contiguous()


def _activations(shape, gen):
    """~ N(0, 1), one channel in a hundred twenty times as large, as hidden states have them."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return (x * (1.0 + 19.0 * (torch.rand(shape[-1:], generator=gen, device=DEV) < 0.01))).bfloat16()


# ------------------------------------------------------------------ prepare --

def _rows(n, E):
    """Rows that hold n choices of E experts in segments of whole 128 rows, whatever the choice; a multiple of 512."""
    return -(-(n + 127 * min(n, E)) // 128 * 128 // 512) * 512


def _choice(T, E, k, padded, gen):
    """A router's choice: some experts sought after, others hardly; the last tokens padding (no expert)."""
    bias = torch.randn(E, generator=gen, device=DEV) * 0.5
    ids = (torch.randn((T, E), generator=gen, device=DEV) + bias).argsort(1, descending=True)[:, :k].int()
    if padded:
        ids[T - padded:] = -1
    w = torch.rand((T, k), generator=gen, device=DEV) + 0.1
    return ids.contiguous(), w / w.sum(1, keepdim=True)


def _buffers(shapes):
    """The output buffers that a training loop keeps: codes of zero, scales of one."""
    return {n: torch.zeros(s, dtype=torch.uint8, device=DEV) if n.startswith("q") else torch.ones(s, device=DEV)
            for n, s in shapes.items()}


def _quantize_buffers(M, C, names):
    shape = {"q": (M, C), "s": (M, C // 128), "qT": (C, M), "sT": (C, M // 128)}
    return _buffers({n: shape[n] for n in names})


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case)
    op, rule = case["op"], case["scale"]
    if op in ("dispatch", "combine"):
        T, E, k, H = (case[n] for n in ("T", "E", "k", "H"))
        s["ids"], s["weights"] = _choice(T, E, k, case["padded"], gen)
        s["R"] = R = _rows(T * k, E)
        if op == "dispatch":
            s["x"] = _activations((T, case["ld"]), gen)[:, :H]
            s["outs"] = _quantize_buffers(R, H, ("q", "s", "qT", "sT") if case["both"] else ("q", "s"))
        else:
            s["rows"], s["source"], s["offsets"] = _plain_sort(s["ids"], E, R)
            s["z"] = randn(R, H).bfloat16()
            if case["back"]:
                s["dy"] = (randn(T, H) * 1e-3).bfloat16()
                s["outs"] = _quantize_buffers(R, H, ("q", "s", "qT", "sT"))
    elif op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        ids, _ = _choice(T, E, k, 0, gen)
        s["R"] = R = _rows(T * k, E)
        _, source, s["offsets"] = _plain_sort(ids, E, R)
        at = s["offsets"].tolist()
        s["segments"] = [(e, at[e], at[e + 1]) for e in range(E)]
        there = (source >= 0)[:, None]
        if case["way"] != "dgrad":
            x = torch.where(there, _activations((R, K), gen).float(), torch.zeros((), device=DEV))
        if case["way"] != "fprop":
            dy = torch.where(there, (randn(R, N) * 1e-3).bfloat16().float(), torch.zeros((), device=DEV))
        if case["way"] == "wgrad":
            s["a"], s["sa"] = _codes_t(dy, rule)
            s["b"], s["sb"] = _codes_t(x, rule)
            s["b"] = s["b"].view(torch.uint8)
            s["out"] = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
        else:
            s["a"], s["sa"] = _codes(x if case["way"] == "fprop" else dy, rule)
            s["b"], s["sb"] = _weight((E, N, K), 0.02, rule, gen)
            s["out"] = torch.zeros((R, N if case["way"] == "fprop" else K), dtype=torch.bfloat16, device=DEV)
        s["a"] = s["a"].view(torch.uint8)
    elif op == "gated":
        M, I = case["M"], case["I"]
        s["gu"] = _activations((M, 2 * I), gen)
        s["limit"] = torch.tensor([case["used"]], dtype=torch.int32, device=DEV)
        s["forward"] = _buffers({"q": (M, I), "s": (M, I // 128), "qc": (M, 2 * I), "sc": (M, 2 * I // 128)})
        if case["back"]:
            s["dh"] = (randn(M, I) * 1e-3).bfloat16()
            s["backward"] = _buffers({"q": (M, 2 * I), "s": (M, 2 * I // 128), "qT": (2 * I, M), "sT": (2 * I, M // 128),
                                      "qhT": (I, M), "shT": (I, M // 128)})
    else:
        M, C = case["M"], case["C"]
        q, s["s"] = _codes(_activations((M, C), gen).float(), rule)
        s["q"] = q.view(torch.uint8)
        s["limit"] = torch.tensor([case["used"]], dtype=torch.int32, device=DEV)
        s["outs"] = _quantize_buffers(M, C, ("qT", "sT"))
    return s


# -------------------------------------------------------------- plain forms --

def _plain_sort(ids, E, R):
    """(the row of each choice, the choice of each row, the segments' starts); -1 where there is none."""
    n = ids.numel()
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add(0, key, torch.ones_like(key))
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    offsets = torch.cat([zero, torch.cumsum((counts[:E] + 127) // 128 * 128, 0)])
    first = torch.cumsum(counts, 0) - counts
    expert = key[order]
    row = torch.where(expert < E, offsets[expert.clamp_max(E - 1)] + torch.arange(n, device=DEV) - first[expert],
                      torch.full_like(expert, -1))
    rows = torch.empty_like(row).scatter(0, order, row)
    source = torch.full((R + 1,), -1, dtype=torch.int64, device=DEV)
    source = source.scatter(0, torch.where(row >= 0, row, torch.full_like(row, R)), order)[:R]
    return rows.view(ids.shape).int(), source.int(), offsets.int()


def _plain_gathered(x, source, k, weights):
    """The sorted rows before they are quantized, fp32."""
    at = source.long().clamp_min(0)
    v = x.float()[at // k]
    if weights is not None:
        v = (v * weights.reshape(-1)[at][:, None]).bfloat16().float()
    return torch.where((source >= 0)[:, None], v, torch.zeros((), device=DEV))


def _plain_both(v, rule, both):
    q, s = _codes(v, rule)
    if not both:
        return {"q": q, "s": s}
    qT, sT = _codes_t(v, rule)
    return {"q": q, "s": s, "qT": qT, "sT": sT}


def _plain_dispatch(s):
    rows, source, offsets = _plain_sort(s["ids"], s["E"], s["R"])
    v = _plain_gathered(s["x"], source, s["k"], None)
    return {"rows": rows, "source": source, "offsets": offsets, **_plain_both(v, s["scale"], s["both"])}


def _plain_combine(s):
    there = s["rows"] >= 0
    z = s["z"].float()[s["rows"].long().clamp_min(0)]  # [T, k, H]
    w = torch.where(there, s["weights"], torch.zeros((), device=DEV))
    y = (z * w[:, :, None]).sum(1)
    r = {"y": y if s["out"] == "fp32" else y.bfloat16()}
    if not s["back"]:
        return r
    dw = (z * s["dy"].float()[:, None, :]).sum(2)
    v = _plain_gathered(s["dy"], s["source"], s["k"], s["weights"])
    return {**r, "dweights": torch.where(there, dw, torch.zeros((), device=DEV)), **_plain_both(v, s["scale"], True)}


def _plain_experts(s):
    out = torch.zeros_like(s["out"])
    a = _value(s["a"], s["sa"])
    b = _value(s["b"], s["sb"]) if s["way"] == "wgrad" else _decode(s["b"], s["sb"])
    for e, lo, hi in s["segments"]:  # a product for each expert
        if s["way"] == "wgrad":
            out[e] = (a[:, lo:hi] @ b[:, lo:hi].t()).bfloat16()
        else:
            out[lo:hi] = (a[lo:hi] @ (b[e].t() if s["way"] == "fprop" else b[e])).bfloat16()
    return out


def _live(q, s, used):
    """Row groups with the rows from `used` on as the buffers held them."""
    live = (torch.arange(q.shape[0], device=DEV) < used)[:, None]
    return (torch.where(live, q.view(torch.uint8), torch.zeros((), dtype=torch.uint8, device=DEV)).view(q.dtype),
            torch.where(live, s, torch.ones((), device=DEV)))


def _live_t(q, s, used):
    rows, groups = torch.arange(q.shape[1], device=DEV), torch.arange(s.shape[1], device=DEV)
    zero = torch.zeros((), dtype=torch.uint8, device=DEV)
    return (torch.where(rows < used, q.view(torch.uint8), zero).view(q.dtype),
            torch.where(groups * 128 < used, s, torch.ones((), device=DEV)))


def _plain_gated(s):
    I, rule, used = s["I"], s["scale"], s["used"]
    gu = s["gu"].float()
    g, u = gu[:, :I], gu[:, I:]
    sig = torch.reciprocal(1.0 + torch.exp2(g * -LOG2E))
    h = (g * sig * u).bfloat16().float()
    q, sc = _live(*_codes(h, rule), used)
    qc, scc = _live(*_codes(gu, rule), used)
    r = {"q": q, "s": sc, "qc": qc, "sc": scc}
    if not s["back"]:
        return r
    kept = _value(qc, scc).bfloat16().float()
    g, u, dh = kept[:, :I], kept[:, I:], s["dh"].float()
    sig = torch.reciprocal(1.0 + torch.exp2(g * -LOG2E))
    silu = g * sig
    h = (silu * u).bfloat16().float()
    dg = dh * u * (sig * (1.0 + g * (1.0 - sig)))
    d = torch.cat([dg, dh * silu], 1).bfloat16().float()
    dq, ds = _live(*_codes(d, rule), used)
    dqT, dsT = _live_t(*_codes_t(d, rule), used)
    qhT, shT = _live_t(*_codes_t(h, rule), used)
    return {**r, "dq": dq, "ds": ds, "dqT": dqT, "dsT": dsT, "qhT": qhT, "shT": shT}


def _plain_requantize(s):
    qT, sT = _live_t(*_codes_t(_value(s["q"], s["s"]).bfloat16().float(), s["scale"]), s["used"])
    return {"qT": qT, "sT": sT}


# ---------------------------------------------------------------------- run --

def _e4m3(q):
    return q.view(torch.float8_e4m3fn)


def run(s):
    if not own:
        return {"dispatch": _plain_dispatch, "combine": _plain_combine, "experts": _plain_experts,
                "gated": _plain_gated, "requantize": _plain_requantize}[s["op"]](s)
    import blockwise_fp8_linear_amd as fb
    mode = fb.FP8BLK_SCALE_FP32 if s["scale"] == FP32 else fb.FP8BLK_SCALE_POW2
    op = s["op"]
    if op == "dispatch":
        rows, source, offsets = fb.fp8_moe_sort(s["ids"], s["E"])
        r = fb.fp8_moe_gather(s["x"], source, s["k"], used=offsets[-1:], transpose=s["both"], scale_mode=mode,
                              **s["outs"])
        names = ("q", "s", "qT", "sT")
        return {"rows": rows, "source": source, "offsets": offsets,
                **{n: _e4m3(t) if n[0] == "q" else t for n, t in zip(names, r)}}
    if op == "combine":
        y = fb.fp8_moe_combine(s["z"], s["rows"], s["weights"],
                               out_dtype=torch.float32 if s["out"] == "fp32" else torch.bfloat16)
        if not s["back"]:
            return {"y": y}
        q, sc, qT, sT, dw = fb.fp8_moe_combine_backward(s["dy"], s["z"], s["rows"], s["source"], s["weights"],
                                                        used=s["offsets"][-1:], scale_mode=mode, **s["outs"])
        return {"y": y, "dweights": dw, "q": _e4m3(q), "s": sc, "qT": _e4m3(qT), "sT": sT}
    if op == "experts":
        f = {"fprop": fb.fp8_moe_gemm_fprop, "dgrad": fb.fp8_moe_gemm_dgrad, "wgrad": fb.fp8_moe_gemm_wgrad}[s["way"]]
        return f(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out=s["out"], scale_mode=mode)
    if op == "gated":
        q, sc, qc, scc = fb.fp8_gated_forward(s["gu"], used=s["limit"], scale_mode=mode, **s["forward"])
        r = {"q": _e4m3(q), "s": sc, "qc": _e4m3(qc), "sc": scc}
        if not s["back"]:
            return r
        dq, ds, dqT, dsT, qhT, shT = fb.fp8_gated_backward(s["dh"], qc, scc, used=s["limit"], scale_mode=mode,
                                                           **s["backward"])
        return {**r, "dq": _e4m3(dq), "ds": ds, "dqT": _e4m3(dqT), "dsT": dsT, "qhT": _e4m3(qhT), "shT": shT}
    qT, sT = fb.fp8_requantize_colgroup(s["q"], s["s"], used=s["limit"], scale_mode=mode, **s["outs"])
    return {"qT": _e4m3(qT), "sT": sT}


def work(case):
    """Each input once and each output once, as far as rows are in use (segments end half a block early on average)."""
    op = case["op"]
    code = 1 + 4 / 128
    if op == "requantize":
        return {"bytes": 2 * code * case["used"] * case["C"], "flops": 4.0 * case["used"] * case["C"]}
    if op == "gated":
        n = case["used"] * case["I"]
        back = (2 + 2 * code + 5 * code) * n if case["back"] else 0
        return {"bytes": (4 + 3 * code) * n + back, "flops": (40.0 if case["back"] else 12.0) * n}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "experts":
        N, K, n = case["N"], case["K"], T * k
        reached = E * (1.0 - (1.0 - k / E) ** T)
        weights = reached * N * K * (code if case["way"] != "wgrad" else 2)
        a, b = (N, K) if case["way"] == "dgrad" else (K, N)
        rows = code * n * a + (code if case["way"] == "wgrad" else 2) * n * b
        return {"bytes": weights + rows, "flops": 2.0 * n * N * K}
    H, live = case["H"], T - case["padded"]
    n = live * k
    reached = E * (1.0 - (1.0 - k / E) ** live)
    rows = n + 63.5 * reached
    if op == "dispatch":
        return {"bytes": 8 * T * k + 4 * _rows(T * k, E) + 2 * live * H + rows * H * code * (2 if case["both"] else 1),
                "flops": 4.0 * n * H}
    y = n * H * 2 + T * H * (4 if case["out"] == "fp32" else 2) + 8 * T * k
    back = n * H * 2 + 2 * live * H + 2 * rows * H * code + 12 * T * k if case["back"] else 0
    return {"bytes": y + back, "flops": (8.0 if case["back"] else 2.0) * n * H}


# -------------------------------------------------------------------- exact --
# The same operators from their definitions in 64 bits, one choice, one expert or one group at a time.

def _two_to(e):
    """2^e in 64 bits, whole numbers e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _byte_value(codes):
    """E4M3 bytes by their fields: (-1)^s 2^(e - 7) (1 + m / 8), and 2^-6 m / 8 where e is 0."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * _two_to(e - 10))
    return torch.where(c >= 128, -v, v)


def _round_e4m3(v):
    """To the nearest E4M3 value, ties to even; |v| <= 448."""
    step = _two_to((torch.frexp(v.abs())[1] - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _exact_codes(x, rule):
    """x float64 [rows, n * 128] -> code values and scales."""
    q = torch.empty_like(x)
    scales = torch.empty((x.shape[0], x.shape[1] // 128), dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[1], 128):
        g = x[:, a:a + 128]
        top = g.abs().amax(1, keepdim=True)
        if rule == FP32:
            s = (top / 448.0).float().double()
            s[top == 0] = 1.0
            v = (g / s).float().double().clamp(-448.0, 448.0)  # the rule's quotient is an fp32 number
        else:
            e = torch.frexp(top / 448.0)[1].clamp_min(-126)  # top / 448 <= 2^e, and > 2^(e - 1) or equal to it
            s = torch.where((top == 448.0 * _two_to(e - 1)) & (e > -126), _two_to(e - 1), _two_to(e))
            s[top == 0] = 1.0
            v = g / s
        q[:, a:a + 128] = _round_e4m3(v)
        scales[:, a // 128] = s[:, 0]
    return q, scales


def _exact_both(x, rule, both):
    q, s = _exact_codes(x, rule)
    if not both:
        return {"q": q, "s": s}
    qT, sT = _exact_codes(x.t().contiguous(), rule)
    return {"q": q, "s": s, "qT": qT, "sT": sT}


def _exact_kept(q, s):
    return q * s.repeat_interleave(128, 1)


def _exact_sort(ids, E, R):
    chosen = [[] for _ in range(E)]
    for c, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            chosen[e].append(c)
    rows, source, offsets = [-1] * ids.numel(), [-1] * R, [0]
    for e in range(E):
        for j, c in enumerate(chosen[e]):
            rows[c], source[offsets[e] + j] = offsets[e] + j, c
        offsets.append(offsets[e] + (len(chosen[e]) + 127) // 128 * 128)
    return [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (rows, source, offsets)]


def _exact_gathered(x, source, k, weights):
    live = torch.nonzero(source >= 0).squeeze(1)
    at = source[live].long()
    v = x.double()[torch.div(at, k, rounding_mode="floor")]
    if weights is not None:
        v = (v * weights.double().flatten()[at, None]).to(torch.bfloat16).double()
    out = torch.zeros((len(source), x.shape[1]), dtype=torch.float64, device=DEV)
    out[live] = v
    return out


def _exact_cut(r, used):
    """Outputs by name, the rows from `used` on as zeros with scales of one."""
    for n, t in r.items():
        codes = n.lstrip("d")[0] == "q"
        if n.endswith("T"):
            t[:, (used if codes else -(-used // 128)):] = 0.0 if codes else 1.0
        else:
            t[used:] = 0.0 if codes else 1.0
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op, rule = case["op"], case["scale"]
    if op == "dispatch":
        rows, source, offsets = _exact_sort(s["ids"], case["E"], s["R"])
        return {"rows": rows.view(case["T"], case["k"]), "source": source, "offsets": offsets,
                **_exact_both(_exact_gathered(s["x"], source, case["k"], None), rule, case["both"])}
    if op == "combine":
        T, H = case["T"], case["H"]
        y = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        dw = torch.zeros((T, case["k"]), dtype=torch.float64, device=DEV)
        for i in range(case["k"]):
            t = torch.nonzero(s["rows"][:, i] >= 0).squeeze(1)
            z = s["z"][s["rows"][t, i].long()].double()
            y[t] += s["weights"][t, i, None].double() * z
            if case["back"]:
                dw[t, i] = torch.einsum("th,th->t", s["dy"][t].double(), z)
        if not case["back"]:
            return {"y": y}
        v = _exact_gathered(s["dy"], s["source"], case["k"], s["weights"])
        return {"y": y, "dweights": dw, **_exact_both(v, rule, True)}
    if op == "experts":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        a = _exact_kept(_byte_value(s["a"]), s["sa"].double())
        if case["way"] == "wgrad":
            b = _exact_kept(_byte_value(s["b"]), s["sb"].double())
        for e, lo, hi in s["segments"]:
            if case["way"] == "wgrad":
                out[e] = a[:, lo:hi] @ b[:, lo:hi].t()
            else:
                w = _byte_value(s["b"][e]) * s["sb"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
                out[lo:hi] = a[lo:hi] @ (w.t() if case["way"] == "fprop" else w)
        return out
    if op == "requantize":
        v = _exact_kept(_byte_value(s["q"]), s["s"].double()).to(torch.bfloat16).double()
        qT, sT = _exact_codes(v.t().contiguous(), rule)
        return _exact_cut({"qT": qT, "sT": sT}, case["used"])
    I = case["I"]
    gu = s["gu"].double()
    h = (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16).double()
    q, sc = _exact_codes(h, rule)
    qc, scc = _exact_codes(gu, rule)
    r = {"q": q, "s": sc, "qc": qc, "sc": scc}
    if case["back"]:
        kept = _exact_kept(qc, scc).to(torch.bfloat16).double()
        g, u, dh = kept[:, :I], kept[:, I:], s["dh"].double()
        sig = torch.sigmoid(g)
        d = torch.cat([dh * u * (sig + g * sig * (1.0 - sig)), dh * g * sig], 1).to(torch.bfloat16).double()
        b = _exact_both(d, rule, True)
        r.update({"d" + n: t for n, t in b.items()})
        r["qhT"], r["shT"] = _exact_codes((g * sig * u).to(torch.bfloat16).double().t().contiguous(), rule)
    return _exact_cut(r, case["used"])
