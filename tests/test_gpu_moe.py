"""fp8_moe_route, its gradient, fp8_moe_experts and fp8_moe_layer against
64-bit references (moe_ref.py), at the sizes and masks where they can go
wrong."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import moe_ref
import oracle
from blockwise_fp8_linear_amd import synth
from gpu_util import dev, dev_bf16, host, host_f32, require_gpu

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# ------------------------------------------------------------------- router --

def _logits(T, E, dtype, seed, masked):
    """Within +-8, with ties (bf16 has few values there), masked entries and rows."""
    rng = synth.rng_for(50, seed)
    v = np.clip(rng.standard_normal((T, E)) * 2.5, -8, 8).astype(np.float32)
    v[rng.random((T, E)) < 0.1] = 0.0
    v[rng.random((T, E)) < 0.05] = -0.0
    if masked:
        v[rng.random((T, E)) < 0.5] = -np.inf
        v[rng.random((T, E)) < 0.05] = np.nan
        v[0] = -np.inf
        if T > 1:
            v[T - 1, 1:] = -np.inf
            v[T - 1, 0] = np.finfo(np.float32).min / 4
    if dtype == "bf16":
        v = (oracle.bf16_rne(v).astype(np.uint32) << 16).view(np.float32)
    return v


def _dev_logits(v, dtype, ld=None):
    import torch
    T, E = v.shape
    wide = torch.full((T, ld or E), 99.0, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    wide[:, :E] = dev(v).to(wide.dtype)
    return wide[:, :E]


ROUTE = [(1, 1, 1), (1, 64, 8), (3, 5, 5), (17, 60, 4), (5, 65, 7), (33, 128, 16), (9, 129, 1), (4, 256, 8),
         (7, 257, 3), (2, 512, 16), (3, 1000, 9), (2, 1024, 16), (1025, 64, 6)]


@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("masked", [False, True])
def test_route_and_gradient(T, E, k, dtype, renorm, masked):
    import torch
    v = _logits(T, E, dtype, T * 2000 + E, masked)
    lg = _dev_logits(v, dtype, ld=E + 3)
    ids, w = fb.fp8_moe_route(lg, k, renormalize=renorm)
    rid, rw = moe_ref.route(v.astype(np.float64), k, renorm)
    assert np.array_equal(host(ids), rid)
    tol = moe_ref.route_tolerance(16, E)
    got = host(w).astype(np.float64)
    assert np.all(np.abs(got - rw) <= tol * rw)
    assert np.all(got[rid < 0] == 0)

    g = synth.rng_for(51, T).standard_normal((T, k)).astype(np.float32)
    wide = torch.full((T, E + 5), 7.0, device="cuda", dtype=lg.dtype)
    d = fb.fp8_moe_route_backward(lg, ids, dev(g), renormalize=renorm, dlogits=wide[:, :E])
    ref = moe_ref.route_backward(v.astype(np.float64), rid, g.astype(np.float64), renorm)
    # dl = p (g - mean): p to tol, the mean a sum of k products
    size = np.abs(g).max() * (1 + k)
    p = np.zeros((T, E))
    for t in range(T):
        row = v[t].astype(np.float64)
        among = [j for j in (rid[t] if renorm else range(E)) if j >= 0 and row[j] > -np.inf]
        for j, q in moe_ref._softmax(row, among).items():
            p[t, j] = q
    lim = p * size * (3 * tol + (k + 4) * moe_ref.U)
    if dtype == "bf16":
        lim = lim + 2.0 ** -8 * np.abs(ref)
    got = host_f32(d).astype(np.float64)
    assert np.all(np.abs(got - ref) <= lim)
    assert bool((wide[:, E:] == 7.0).all()), "wrote past the row"
    d2 = fb.fp8_moe_route_backward(lg, ids, dev(g), renormalize=renorm)
    assert torch.equal(d2, d)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    """d sum(g w) / d logits by central differences of the 64-bit weights at a
    point without ties (the choice does not change within the step)."""
    T, E, k = 5, 12, 4
    rng = synth.rng_for(52, int(renorm))
    v = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) * 0.37 - 2.0
    g = rng.standard_normal((T, k)).astype(np.float32)
    ids, _ = fb.fp8_moe_route(dev(v), k, renormalize=renorm)
    d = host(fb.fp8_moe_route_backward(dev(v), ids, dev(g), renormalize=renorm)).astype(np.float64)
    step = 1e-4
    num = np.zeros((T, E))
    for j in range(E):
        up, down = v.astype(np.float64), v.astype(np.float64)
        up[:, j] += step
        down[:, j] -= step
        num[:, j] = ((moe_ref.route(up, k, renorm)[1] - moe_ref.route(down, k, renorm)[1]) * g).sum(1) / (2 * step)
    # third derivatives of a softmax weight are below 1: step^2 / 6 of sum |g|, and fp32 on the kernel's side
    lim = np.abs(g).sum(1, keepdims=True) * (step ** 2 + moe_ref.route_tolerance(8, E) * 4)
    assert np.all(np.abs(d - num) <= lim)


def test_route_more_tokens_than_a_launch():
    import torch
    T, tail = 2 ** 24 + 5, slice(-40, None)
    lg = torch.randn((T, 3), device="cuda", dtype=torch.bfloat16)
    lg[5] = -torch.inf
    ids, w = fb.fp8_moe_route(lg, 2, renormalize=False)
    assert int(ids[5].max()) == -1
    first = lg.float().argmax(1)                             # (of equal ones any)
    rest = torch.arange(T, device="cuda") != 5
    assert bool((lg.gather(1, ids.long().clamp(min=0))[:, 0] == lg.gather(1, first[:, None])[:, 0])[rest].all())
    g = torch.randn((T, 2), device="cuda")
    d = fb.fp8_moe_route_backward(lg, ids, g, renormalize=False)
    alone = fb.fp8_moe_route(lg[tail], 2, renormalize=False)
    assert torch.equal(ids[tail], alone[0]) and torch.equal(w[tail], alone[1])
    assert torch.equal(d[tail], fb.fp8_moe_route_backward(lg[tail], *(t[tail] for t in (ids, g)), renormalize=False))


def test_route_infinities_and_lowest():
    inf, low = np.inf, np.finfo(np.float32).min
    v = np.array([[inf, 1.0, inf, 0.0], [low, low, low, low], [low, 3.4e38, 0.0, -inf], [np.nan, inf, -inf, np.nan]],
                 np.float32)
    ids, w = fb.fp8_moe_route(dev(v), 3)
    assert host(ids).tolist() == [[0, 2, 1], [0, 1, 2], [1, 2, 0], [1, -1, -1]]
    assert np.array_equal(host(w)[[0, 2, 3]], np.array([[.5, .5, 0], [1, 0, 0], [1, 0, 0]], np.float32))
    assert np.all(np.abs(host(w)[1] - 1 / 3) <= 2.0 ** -24)
    ids, w = fb.fp8_moe_route(dev(v), 2, renormalize=False)
    assert host(ids).tolist() == [[0, 2], [0, 1], [1, 2], [1, -1]]
    assert np.array_equal(host(w), np.array([[.5, .5], [.25, .25], [1, 0], [1, 0]], np.float32))
    d = host(fb.fp8_moe_route_backward(dev(v), ids, dev(np.ones((4, 2), np.float32)), renormalize=False))
    # row 1: p = 1/4 each, two chosen with g = 1: mean 1/2
    assert np.array_equal(d, np.array([[0] * 4, [.125, .125, -.125, -.125], [0] * 4, [0] * 4], np.float32))


def test_route_backward_ids_that_are_none_or_twice():
    v = synth.rng_for(53).standard_normal((3, 6)).astype(np.float32)
    ids = np.array([[2, -1, 5], [4, 4, 1], [6, 1000, -7]], np.int32)
    g = np.array([[1.0, np.nan, -2.0], [0.5, 0.25, 1.0], [np.inf, 1.0, 2.0]], np.float32)
    for renorm in (True, False):
        d = host(fb.fp8_moe_route_backward(dev(v), dev(ids), dev(g), renormalize=renorm)).astype(np.float64)
        ref = moe_ref.route_backward(v.astype(np.float64), ids, g.astype(np.float64), renorm)
        assert np.all(np.abs(d - ref) <= 4 * moe_ref.route_tolerance(8, 6))


# ------------------------------------------------------------------ experts --

def _weights(E, rows, cols, std, key, mode):
    w = synth.normal_bf16((E * rows, cols), std, 54, key)
    q, _, s = oracle.quantize_block(w, transpose=False, mode=mode)
    return q.reshape(E, rows, cols), s.reshape(E, rows // 128, cols // 128)


def _case(T, H, I, E, k, seed, mode, ids=None):
    rng = synth.rng_for(55, seed)
    x = synth.normal_bf16((T, H), 1.0, 55, seed, 1)
    w1, w2 = _weights(E, 2 * I, H, 0.05, seed * 2, mode), _weights(E, H, I, 0.05, seed * 2 + 1, mode)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = (rng.random((T, ids.shape[1])) + 0.1).astype(np.float32)
    return x, ids, w, *w1, *w2


EXPERTS = [(1, 256, 128, 4, 2), (1, 128, 384, 16, 16), (2, 384, 256, 3, 3), (15, 256, 128, 5, 2), (16, 128, 128, 8, 4),
           (17, 256, 256, 4, 1), (31, 128, 128, 2, 2), (33, 384, 128, 6, 3), (64, 256, 384, 3, 2), (65, 128, 128, 1, 1),
           (130, 256, 128, 2, 1), (200, 128, 256, 40, 5), (512, 128, 128, 3, 2),
           (20, 384, 128, 40, 2), (20, 128, 256, 64, 4), (12, 128, 512, 64, 8), (6, 128, 768, 64, 8),
           (40, 128, 128, 1024, 16)]


@pytest.mark.parametrize("T,H,I,E,k", EXPERTS)
@pytest.mark.parametrize("mode", [POW2, FP32])
def test_experts(T, H, I, E, k, mode):
    import torch
    x, ids, w, q1, s1, q2, s2 = _case(T, H, I, E, k, T + E, mode)
    if T > 2:
        ids[T // 2] = -1                         # a padded token
        ids[0, 0] = E                            # an id past the experts
        ids[1, k - 1] = np.iinfo(np.int32).min
    ref, bound = moe_ref.experts(x, ids, w, q1, s1, q2, s2, mode)
    wide = torch.zeros((T, H + 24), device="cuda", dtype=torch.bfloat16)
    wide[:, :H] = dev_bf16(x)
    args = (wide[:, :H], dev(ids), dev(w), dev(q1), dev(s1), dev(q2), dev(s2))
    y32 = fb.fp8_moe_experts(*args, out_dtype=torch.float32, scale_mode=mode)
    got = host(y32).astype(np.float64)
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)))
    if T > 2:
        assert np.all(got[T // 2] == 0)
    y = fb.fp8_moe_experts(*args, scale_mode=mode)
    assert torch.equal(y, y32.bfloat16())        # the same sums, rounded once
    assert torch.equal(fb.fp8_moe_experts(*args, out_dtype=torch.float32, scale_mode=mode), y32)


def _exact_case(T, E, k, seed, H=256, I=256, ids=None):
    """Whole numbers throughout: g = 32 or 64 exactly (its silu rounds to
    itself), u whole and at most 12, so every rounding on the way is exact and
    y is a whole number below 2^24."""
    rng = synth.rng_for(56, seed)
    x = rng.integers(-3, 4, (T, H)).astype(np.float32)
    x[:, 0] = 1.0
    G = np.zeros((E, I, H), np.float32)
    G[:, :, 0] = rng.choice([32.0, 64.0], (E, I))
    Uw = np.zeros((E, I, H), np.float32)
    for n in range(4):
        np.put_along_axis(Uw, rng.integers(1, H, (E, I, 1)), rng.choice([-1.0, 1.0], (E, I, 1)), axis=2)
    Wd = rng.integers(-1, 2, (E, H, I)).astype(np.float32)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.choice([0.5, 1.0, 2.0], (T, k)).astype(np.float32)
    bits = lambda a: oracle.bf16_rne(a.reshape(-1, a.shape[-1]))  # noqa: E731
    q1, _, s1 = oracle.quantize_block(bits(np.concatenate([G, Uw], 1)), transpose=False)
    q2, _, s2 = oracle.quantize_block(bits(Wd), transpose=False)
    y = np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            y[t] += float(w[t, j]) * (Wd[e].astype(np.float64) @ ((G[e] @ x[t]).astype(np.float64) * (Uw[e] @ x[t])))
    return (dev_bf16(bits(x)), dev(ids), dev(w), dev(q1.reshape(E, 2 * I, H)),
            dev(s1.reshape(E, 2 * I // 128, H // 128)), dev(q2.reshape(E, H, I)),
            dev(s2.reshape(E, H // 128, I // 128))), y


@pytest.mark.parametrize("T,E,k", [(1, 3, 2), (7, 9, 4), (16, 2, 2), (40, 5, 3), (100, 1, 1), (300, 4, 2)])
def test_experts_exact(T, E, k):
    import torch
    args, y = _exact_case(T, E, k, T)
    assert np.array_equal(host(fb.fp8_moe_experts(*args, out_dtype=torch.float32)).astype(np.float64), y)


@pytest.mark.parametrize("T,E", [(14, 16), (40, 8), (200, 16), (512, 32)])
def test_experts_one_has_all_the_tokens(T, E):
    """Many times the rows that an expert has on average."""
    import torch
    ids = np.tile(np.array([[3, 5]], np.int32), (T, 1))
    ids[T // 2:, 1] = -1
    ids[0] = [6, 3]
    args, y = _exact_case(T, E, 2, 900 + T, ids=np.maximum(ids, 0))
    assert np.array_equal(host(fb.fp8_moe_experts(*args, out_dtype=torch.float32)).astype(np.float64), y)
    want = fb.fp8_moe_experts(args[0], dev(ids), *args[2:], out_dtype=torch.float32)
    alone = [fb.fp8_moe_experts(args[0][t:t + 1], dev(ids[t:t + 1]), args[2][t:t + 1], *args[3:],
                                out_dtype=torch.float32) for t in (0, 1, T - 1)]
    assert torch.equal(want[[0, 1, T - 1]], torch.cat(alone))


@pytest.mark.parametrize("T,H,I,E,k", [(8, 4096, 512, 32, 8), (3, 8960, 256, 3, 2), (3, 256, 8448, 3, 2),
                                       (20, 8960, 256, 5, 2), (20, 256, 8448, 5, 2), (20, 384, 8448, 3, 3),
                                       (14, 256, 8448, 4, 2), (70, 8448, 128, 2, 1)])
def test_experts_exact_long(T, H, I, E, k):
    """Reductions longer than the scales that are kept at a time, and long
    enough for several workgroups to share a column."""
    import torch
    args, y = _exact_case(T, E, k, 500 + T, H, I)
    assert np.abs(y).max() < 2 ** 24
    assert np.array_equal(host(fb.fp8_moe_experts(*args, out_dtype=torch.float32)).astype(np.float64), y)


def test_experts_same_expert_twice_and_none():
    """An expert named twice by a token counts twice; a batch that reaches no
    expert at all gives zeros."""
    import torch
    for T in (3, 30):
        args, _ = _exact_case(T, 4, 2, 90 + T)
        x, ids, w = args[:3]
        once = fb.fp8_moe_experts(x, ids[:, :1].contiguous(), w[:, :1].contiguous(), *args[3:], out_dtype=torch.float32)
        twice = fb.fp8_moe_experts(x, ids[:, :1].expand(-1, 2).contiguous(), w[:, :1].expand(-1, 2).contiguous(),
                                   *args[3:], out_dtype=torch.float32)
        assert torch.equal(twice, 2 * once)
        none = fb.fp8_moe_experts(x, torch.full_like(ids, -1), w, *args[3:], out=torch.full_like(x, 5.0))
        assert bool((none == 0).all())


@pytest.mark.parametrize("T", [5, 50])
def test_experts_one_token_does_not_reach_another(T):
    """Infinities and NaN of one token (in its row, or in an expert that only
    it chose) stay in its row."""
    import torch
    args, _ = _exact_case(T, 4, 2, 70 + T)
    x, ids, w = args[0].clone(), args[1].clone(), args[2]
    ids[:] = torch.randint(0, 3, ids.shape, device="cuda", dtype=torch.int32)
    ids[2] = 3
    clean = fb.fp8_moe_experts(x, ids, w, *args[3:], out_dtype=torch.float32)
    x[2, 7], x[2, 200] = float("inf"), float("nan")
    q1, q2 = args[3].clone(), args[5].clone()
    q1[3, 5, 3], q2[3, 9, 1] = 0x7F, 0xFF        # NaN codes
    y = fb.fp8_moe_experts(x, ids, w, q1, args[4], q2, args[6], out_dtype=torch.float32)
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[2]).any())


# ------------------------------------------------------------ a whole layer --

@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (6, 384, 128, 17, 3), (16, 128, 256, 4, 4),
                                       (20, 256, 128, 70, 8), (100, 128, 128, 9, 2), (3, 1024, 128, 70, 5),
                                       (20, 1024, 128, 70, 5), (12, 640, 128, 20, 3)])
@pytest.mark.parametrize("renorm", [True, False])
def test_layer_is_route_and_experts(T, H, I, E, k, renorm):
    import torch
    x, _, _, q1, s1, q2, s2 = _case(T, H, I, E, 1, 300 + T, POW2)
    wr = synth.normal_bf16((E, H), 0.3, 57, T)
    exps = tuple(dev(a) for a in (q1, s1, q2, s2))
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), dtype=torch.float32, device="cuda")
    y = fb.fp8_moe_layer(dev_bf16(x), dev_bf16(wr), *exps, k, renormalize=renorm, ids=ids, weights=w,
                         out_dtype=torch.float32)
    # the logits are fp32 sums: experts closer than their error may change places, so each choice is held to the
    # logit that belongs there, and the weights to the softmax of what was chosen
    lg = moe_ref.f64(x) @ moe_ref.f64(wr).T
    err = (H + 16) * 2 * moe_ref.U * (np.abs(moe_ref.f64(x)) @ np.abs(moe_ref.f64(wr)).T).max()
    got, gw = host(ids), host(w).astype(np.float64)
    for t in range(T):
        row, chosen = lg[t], list(got[t])
        assert len(set(chosen)) == k
        assert np.all(np.abs(row[chosen] - np.sort(row)[::-1][:k]) <= 2 * err)
        p = moe_ref._softmax(row, chosen if renorm else list(range(E)))
        rw = np.array([p[j] for j in chosen])
        assert np.all(np.abs(gw[t] - rw) <= (2 * err + moe_ref.route_tolerance(np.ptp(lg), E)) * 1.01 * rw)
    # the layer is its parts: the same choice through the experts gives the same bits
    assert torch.equal(y, fb.fp8_moe_experts(dev_bf16(x), ids, w, *exps, out_dtype=torch.float32))
    assert torch.equal(fb.fp8_moe_layer(dev_bf16(x), dev_bf16(wr), *exps, k, renormalize=renorm), y.bfloat16())


def test_all_together_in_a_graph():
    """A decoding step as it would run -- a projection of a few tokens, the
    layer, the projection back -- captured once and replayed, with other work
    between the replays; two graphs share one workspace."""
    import torch
    H, I, E, k = 256, 128, 12, 3
    graphs = []
    ws = torch.empty(max(fb.fp8_moe_workspace_size(t, H, I, E, k) for t in (4, 33)), dtype=torch.uint8, device="cuda")
    for T in (4, 33):
        x, _, _, q1, s1, q2, s2 = _case(T, H, I, E, 1, 400 + T, POW2)
        wr, wo = dev_bf16(synth.normal_bf16((E, H), 0.3, 58, T)), dev_bf16(synth.normal_bf16((H, H), 0.05, 59, T))
        qo, _, so = fb.fp8_quantize_block(wo, transpose=False)
        exps = tuple(dev(a) for a in (q1, s1, q2, s2))
        x = dev_bf16(x)
        a, b, c = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(3))

        def step(x=x, a=a, b=b, c=c, qo=qo, so=so, wr=wr, exps=exps):
            fb.fp8_linear(x, qo, so, out=a)
            fb.fp8_moe_layer(a, wr, *exps, k, out=b, workspace=ws)
            fb.fp8_linear(b, qo, so, out=c)

        step()
        torch.cuda.synchronize()
        ref = c.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, c, b, ref, step))         # step keeps the graph's inputs alive
    other = torch.randn(256, 256, device="cuda")
    for _ in range(3):
        for g, c, b, ref, _ in graphs:
            c.fill_(3.0)
            b.fill_(-1.0)
            ws.fill_(0xFF)
            other = other @ other.T / 256
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c, ref)


def test_on_another_stream():
    import torch
    args, y = _exact_case(9, 4, 2, 777)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fb.fp8_moe_experts(*args, out_dtype=torch.float32, stream=s)
    ids, w = fb.fp8_moe_route(dev(np.arange(12, dtype=np.float32).reshape(2, 6)), 2, stream=s)
    s.synchronize()
    assert np.array_equal(host(got).astype(np.float64), y)
    assert host(ids).tolist() == [[5, 4], [5, 4]]
