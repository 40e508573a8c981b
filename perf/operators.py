"""The operators that carry the FP8 linear layer from training batches to any
number of tokens and to mixtures of experts, as they are measured.

  linear   fp8_linear: y = x W^T for any number of tokens; x bf16, quantized
           in groups of 128 on the way, W in E4M3 blocks of 128 x 128.
  route    fp8_moe_route (and fp8_moe_route_backward): the top-k experts of
           each token's router logits, their softmax weights, the gradient.
  moe      fp8_moe_layer / fp8_moe_experts: a whole mixture-of-experts layer
           for a few tokens, the experts' weights in E4M3 blocks.

`run` computes them in elementary torch operations where `own` is false and
by the library's entry points where it is true.  Rounding, on both sides as
the library documents it: activations to E4M3 right before each product (one
scale per 128 values), the gated product of an expert to bf16 once before
that, results to the output type once; everything else in 32 bits or more.
"""
import math

import torch

own = False

DEV = "cuda"
POW2, FP32 = "pow2", "amax448"


# -------------------------------------------------------------------- cases --

def listed():
    return [
        # the decoder layer's linears (hidden 2048, 16 + 2 x 8 heads of 128, MLP 6144) while serving:
        # one sequence's next token through the QKV projection -- latency, nothing but the weights to read
        dict(name="linear 1 qkv", op="linear", M=1, N=4096, K=2048, ld=2048, out="bf16", scale=POW2),
        # a handful of sequences through the down projection, result kept in fp32 for a residual stream
        dict(name="linear 7 down fp32", op="linear", M=7, N=2048, K=6144, ld=6144, out="fp32", scale=POW2),
        # a serving batch through gate/up; x is a column slice of a wider buffer; amax / 448 scales
        dict(name="linear 48 gate/up", op="linear", M=48, N=12288, K=2048, ld=4096, out="bf16", scale=FP32),
        # a short odd prompt through the attention output projection
        dict(name="linear 333 o", op="linear", M=333, N=2048, K=2048, ld=2048, out="bf16", scale=POW2),
        # a long odd prompt through the QKV projection: bound by the matrix cores
        dict(name="linear 4133 qkv", op="linear", M=4133, N=4096, K=2048, ld=2048, out="bf16", scale=POW2),
        # routing a few tokens while serving: pure latency
        dict(name="route 5", op="route", T=5, E=64, k=6, dtype="bf16", renorm=True, masked=0.0, back=False),
        # routing a ragged micro-batch while training, some experts masked out, some rows with none left
        dict(name="route 4095 masked", op="route", T=4095, E=60, k=4, dtype="bf16", renorm=True, masked=0.3, back=True),
        # routing a whole micro-batch of 4 x 4096 while training, weights of the full softmax, with the gradient
        dict(name="route 16384", op="route", T=16384, E=128, k=8, dtype="fp32", renorm=False, masked=0.0, back=True),
        # one sequence's next token through many small experts
        dict(name="moe 1 of 64", op="moe", T=1, E=64, k=8, H=2048, I=1024, router=True, padded=0, scale=POW2),
        # a few sequences through few large experts, routed by the caller, the batch padded at its end
        dict(name="moe 9 of 8 padded", op="moe", T=9, E=8, k=2, H=2048, I=6144, router=False, padded=2, scale=POW2),
        # a serving batch through many smaller experts, amax / 448 scales
        dict(name="moe 40 of 128", op="moe", T=40, E=128, k=8, H=2048, I=768, router=True, padded=0, scale=FP32),
        # a large serving batch: every expert is read, and each has dozens of tokens
        dict(name="moe 256 of 64", op="moe", T=256, E=64, k=8, H=2048, I=1024, router=True, padded=0, scale=POW2),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "moe", "moe"])
    scale = rng.choice([POW2, POW2, FP32])
    if op == "linear":
        M, N, K = _log(rng, 1, 4096), 128 * _log(rng, 1, 96), 128 * _log(rng, 1, 64)
        while M * N * K > 4096 * 4096 * 2048:
            M //= 2
        # fp32 results are a small batch's; a long prompt's are bf16, the type of the activations
        out = rng.choice(["bf16", "fp32"]) if M <= 64 else "bf16"
        return dict(op=op, M=M, N=N, K=K, ld=K + 8 * rng.choice([0, 0, 1, 33]), out=out, scale=scale)
    if op == "route":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 16000), E=E, k=rng.randint(1, min(8, E)), dtype=rng.choice(["bf16", "fp32"]),
                    renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.2, 0.6]), back=rng.random() < 0.6)
    T, E, H, I = _log(rng, 1, 256), _log(rng, 4, 128), 128 * _log(rng, 2, 32), 128 * _log(rng, 1, 48)
    while E * H * I > 64 * 2048 * 1024:
        E, I = (E // 2, I) if E >= 8 else (E, I // 256 * 128)
    router = rng.random() < 0.6
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), H=H, I=I, router=router,
                padded=0 if router else rng.randint(0, T // 2), scale=scale)


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


def _quantize(x, rule):
    """x fp32 [rows, K] -> the values its E4M3 codes stand for, scales applied (fp32: a code times its scale is exact
    under the power-of-two rule and rounded once under the other)."""
    g = x.view(x.shape[0], -1, 128)
    s = _scales(g.abs().amax(2, keepdim=True), rule)
    q = (g / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * s).view_as(x)


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

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rand = lambda *shape: torch.rand(shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case)
    if case["op"] == "linear":
        wide = _activations((case["M"], case["ld"]), gen)
        s["x"] = wide[:, :case["K"]]
        s["qw"], s["sw"] = _weight((case["N"], case["K"]), 0.02, case["scale"], gen)
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn((T, E), generator=gen, device=DEV) * 1.5
        if case["masked"]:
            logits[rand(T, E) < case["masked"]] = -math.inf
            logits[rand(T) < 0.01] = -math.inf  # and a few rows that keep nothing
        s["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["dweights"] = torch.randn((T, case["k"]), generator=gen, device=DEV)
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = _activations((T, H), gen)
        s["qw1"], s["sw1"] = _weight((E, 2 * I, H), 0.02, case["scale"], gen)
        s["qw2"], s["sw2"] = _weight((E, H, I), 0.02, case["scale"], gen)
        if case["router"]:
            s["wr"] = (torch.randn((E, H), generator=gen, device=DEV) * 0.02).bfloat16()
        else:
            s["ids"] = rand(T, E).argsort(1)[:, :k].int()
            w = rand(T, k) + 0.1
            s["weights"] = w / w.sum(1, keepdim=True)
            if case["padded"]:
                s["ids"][T - case["padded"]:] = -1
            s["ids"] = s["ids"].contiguous()
    return s


# -------------------------------------------------------------- plain forms --

def _plain_linear(s):
    y = _quantize(s["x"].float(), s["scale"]) @ _decode(s["qw"], s["sw"]).t()
    return y if s["out"] == "fp32" else y.bfloat16()


def _plain_choose(logits, k):
    """The k largest logits of each row, ties to the lowest index; -inf (and NaN) are not to be chosen.  (ids, with -1
    where nothing is left; which of them are there)."""
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    there = torch.gather(logits, 1, order) > -math.inf
    return torch.where(there, order, torch.full_like(order, -1)).int(), there


def _plain_softmax(logits, ids, there, renorm):
    """Softmax weights of the chosen experts (fp32) and the probabilities [T, E] they come from."""
    if renorm:
        keep = torch.zeros_like(logits).scatter_add(1, ids.long().clamp_min(0), there.to(logits.dtype)) > 0
        logits = torch.where(keep, logits, torch.full_like(logits, -math.inf))
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    p = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    return torch.where(there, torch.gather(p, 1, ids.long().clamp_min(0)), torch.zeros((), device=DEV)), p


def _plain_route(s):
    logits = s["logits"].float()
    ids, there = _plain_choose(logits, s["k"])
    weights, p = _plain_softmax(logits, ids, there, s["renorm"])
    if not s["back"]:
        return {"ids": ids, "weights": weights}
    g = torch.where(there, s["dweights"], torch.zeros((), device=DEV))
    full = torch.zeros_like(logits).scatter_add(1, ids.long().clamp_min(0), g)
    dlogits = p * (full - (g * weights).sum(1, keepdim=True))
    return {"ids": ids, "weights": weights, "dlogits": dlogits.to(s["logits"].dtype)}


def _plain_moe(s):
    T, E, I = s["T"], s["E"], s["I"]
    x = s["x"]
    if s["router"]:
        logits = (x.double() @ s["wr"].double().t()).float()  # 64 bits: which expert is chosen hangs on it
        ids, there = _plain_choose(logits, s["k"])
        weights, _ = _plain_softmax(logits, ids, there, True)
    else:
        ids, weights = s["ids"], s["weights"]
        there = ids >= 0
    share = torch.zeros((T, E), device=DEV).scatter_add(1, ids.long().clamp_min(0),
                                                        torch.where(there, weights, torch.zeros((), device=DEV)))
    gu = (_quantize(x.float(), s["scale"]) @ _decode(s["qw1"], s["sw1"]).flatten(0, 1).t()).view(T, E, 2 * I)
    g, u = gu[..., :I], gu[..., I:]
    h = (g / (1.0 + torch.exp(-g)) * u).bfloat16().float()
    h = _quantize(h.reshape(T * E, I), s["scale"]).view(T, E, I) * share[..., None]
    w2 = _decode(s["qw2"], s["sw2"]).transpose(0, 1).reshape(s["H"], E * I)
    return (h.view(T, E * I) @ w2.t()).bfloat16()


# ---------------------------------------------------------------------- run --

def run(s):
    if not own:
        return {"linear": _plain_linear, "route": _plain_route, "moe": _plain_moe}[s["op"]](s)
    import blockwise_fp8_linear_amd as fb
    if s["op"] == "route":
        ids, weights = fb.fp8_moe_route(s["logits"], s["k"], renormalize=s["renorm"])
        if not s["back"]:
            return {"ids": ids, "weights": weights}
        dlogits = fb.fp8_moe_route_backward(s["logits"], ids, s["dweights"], renormalize=s["renorm"])
        return {"ids": ids, "weights": weights, "dlogits": dlogits}
    mode = fb.FP8BLK_SCALE_FP32 if s["scale"] == FP32 else fb.FP8BLK_SCALE_POW2
    if s["op"] == "linear":
        return fb.fp8_linear(s["x"], s["qw"], s["sw"], scale_mode=mode,
                             out_dtype=torch.float32 if s["out"] == "fp32" else torch.bfloat16)
    if s["router"]:
        return fb.fp8_moe_layer(s["x"], s["wr"], s["qw1"], s["sw1"], s["qw2"], s["sw2"], s["k"], scale_mode=mode)
    return fb.fp8_moe_experts(s["x"], s["ids"], s["weights"], s["qw1"], s["sw1"], s["qw2"], s["sw2"], scale_mode=mode)


def work(case):
    """Each input once and each output once; of the experts' weights those that the tokens reach, in expectation."""
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": 2 * M * K + N * K + N * K / 128 ** 2 * 4 + out * M * N, "flops": 2.0 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        back = T * E * size + T * k * 4 if case["back"] else 0
        return {"bytes": T * E * size + T * k * 8 + back, "flops": (8.0 if case["back"] else 4.0) * T * E}
    H, I, T = case["H"], case["I"], T - case["padded"]
    reached = E * (1.0 - (1.0 - k / E) ** T)
    route = 2 * E * H if case["router"] else 8 * T * k
    return {"bytes": reached * 3 * H * I * (1 + 4 / 128 ** 2) + 4 * T * H + route,
            "flops": 6.0 * T * k * H * I + (2.0 * T * E * H if case["router"] else 0)}


# -------------------------------------------------------------------- exact --
# The same operators from their definitions in 64 bits, one token or one expert at a time where that is plainest.

def _two_to(e):
    """2^e in 64 bits, whole numbers e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _value(codes):
    """E4M3 bytes by their fields: (-1)^s 2^(e - 7) (1 + m / 8), and 2^-6 m / 8 where e is 0."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * _two_to(e - 10))
    return torch.where(c >= 128, -v, v)


def _round_e4m3(v):
    """To the nearest E4M3 value, ties to even; |v| <= 448."""
    step = _two_to((torch.frexp(v.abs())[1] - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _exact_quantize(x, rule):
    out = torch.empty_like(x)
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
        out[:, a:a + 128] = _round_e4m3(v) * s
    return out


def _exact_weight(q, s):
    return _value(q) * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _exact_row(row, k, renorm):
    """One token's choice: (ids, weights, and the probabilities that they and the gradient come from)."""
    left = [j for j in range(len(row)) if row[j] > -math.inf]
    chosen = sorted(left, key=lambda j: (-row[j], j))[:k]
    among = chosen if renorm else left
    top = max((row[j] for j in among), default=0.0)
    z = math.fsum(math.exp(row[j] - top) for j in among)
    return chosen, {j: math.exp(row[j] - top) / z for j in among}


def _exact_route(s, logits, k, renorm):
    rows = logits.double().cpu().tolist()
    ids = torch.full((len(rows), k), -1, dtype=torch.int32)
    weights = torch.zeros((len(rows), k), dtype=torch.float64)
    back = "dweights" in s and s["back"]
    dlogits = torch.zeros((len(rows), len(rows[0])), dtype=torch.float64)
    given = s["dweights"].double().cpu().tolist() if back else None
    for t, row in enumerate(rows):
        chosen, p = _exact_row(row, k, renorm)
        for i, j in enumerate(chosen):
            ids[t, i], weights[t, i] = j, p[j]
        if back:
            # w_i = p(chosen_i); dw_i/dl_j = p_i ([i = j] - p_j)
            mean = math.fsum(given[t][i] * p[j] for i, j in enumerate(chosen))
            at = {j: given[t][i] for i, j in enumerate(chosen)}
            out = [0.0] * len(row)
            for j in p:
                out[j] = p[j] * (at.get(j, 0.0) - mean)
            dlogits[t] = torch.tensor(out, dtype=torch.float64)
    return ids.to(DEV), weights.to(DEV), dlogits.to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_quantize(s["x"].double(), case["scale"]) @ _exact_weight(s["qw"], s["sw"]).t()
    if case["op"] == "route":
        ids, weights, dlogits = _exact_route(s, s["logits"], case["k"], case["renorm"])
        r = {"ids": ids, "weights": weights}
        return {**r, "dlogits": dlogits} if case["back"] else r
    x, I = s["x"].double(), case["I"]
    if case["router"]:
        ids, weights, _ = _exact_route(s, x @ s["wr"].double().t(), case["k"], True)
    else:
        ids, weights = s["ids"], s["weights"].double()
    qx = _exact_quantize(x, case["scale"])
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        t, i = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gu = qx[t] @ _exact_weight(s["qw1"][e], s["sw1"][e]).t()
            g, u = gu[:, :I], gu[:, I:]
            h = _exact_quantize((g * torch.sigmoid(g) * u).to(torch.bfloat16).double(), case["scale"])
            y.index_add_(0, t, weights[t, i, None] * (h @ _exact_weight(s["qw2"][e], s["sw2"][e]).t()))
    return y
