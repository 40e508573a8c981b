"""The operators of include/fp8train.h together, as one training step of a
mixture-of-experts layer uses them: against the layer without quantization in 64
bits, in captured graphs, on streams of their own and on two at once."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
from blockwise_fp8_linear_amd import synth
from gpu_util import dev_bf16, host, require_gpu
from train_ref import f64

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
MODES = pytest.mark.parametrize("mode", [POW2, FP32])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Layer:
    """A layer's weights, quantized, and one batch."""

    def __init__(self, T, H, I, E, k, mode, key, renormalize=True):
        self.T, self.H, self.I, self.E, self.k, self.mode, self.renormalize = T, H, I, E, k, mode, renormalize
        self.w1 = synth.normal_bf16((E * 2 * I, H), H ** -0.5, 801, key)
        self.w2 = synth.normal_bf16((E * H, I), I ** -0.5, 802, key)
        q1, _, s1 = fb.fp8_quantize_block(dev_bf16(self.w1), transpose=False, scale_mode=mode)
        q2, _, s2 = fb.fp8_quantize_block(dev_bf16(self.w2), transpose=False, scale_mode=mode)
        self.q1, self.s1 = q1.view(E, 2 * I, H), s1.view(E, 2 * I // 128, H // 128)
        self.q2, self.s2 = q2.view(E, H, I), s2.view(E, H // 128, I // 128)
        self.batch(key)

    def batch(self, key):
        self.x = synth.normal_bf16((self.T, self.H), 1.0, 803, key)
        self.logits = synth.normal_bf16((self.T, self.E), 2.0, 804, key)
        self.logits[self.T // 2] = 0xFF80                   # -infinity: a token with no expert
        if self.E > 2:
            self.logits[: self.T // 4, 1] = 0xFF80          # and an expert masked out for some
        self.dy = synth.normal_bf16((self.T, self.H), 1e-3, 805, key)

    def device(self):
        return [dev_bf16(t) for t in (self.x, self.logits, self.dy)]

    def step(self, x, logits, dy, stream=None):
        """Forward and backward: (y, dx, dlogits, dw1, dw2)."""
        import torch
        kw = dict(stream=stream, scale_mode=self.mode)
        ids, weights = fb.fp8_moe_route(logits, self.k, renormalize=self.renormalize, stream=stream)
        rows, source, offsets = fb.fp8_moe_sort(ids, self.E, stream=stream)
        used = offsets[-1:]
        qx, sx = fb.fp8_moe_gather(x, source, self.k, used=used, **kw)
        gu = fb.fp8_moe_gemm_fprop(qx, sx, self.q1, self.s1, offsets, **kw)
        qh, sh, qc, sc = fb.fp8_gated_forward(gu, used=used, **kw)
        z = fb.fp8_moe_gemm_fprop(qh, sh, self.q2, self.s2, offsets, **kw)
        y = fb.fp8_moe_combine(z, rows, weights, stream=stream)
        del gu, qh, sh
        qz, sz, qzT, szT, dweights = fb.fp8_moe_combine_backward(dy, z, rows, source, weights, used=used, **kw)
        dh = fb.fp8_moe_gemm_dgrad(qz, sz, self.q2, self.s2, offsets, **kw)
        qg, sg, qgT, sgT, qhT, shT = fb.fp8_gated_backward(dh, qc, sc, used=used, **kw)
        dw2 = fb.fp8_moe_gemm_wgrad(qzT, szT, qhT, shT, offsets, out_dtype=torch.float32, **kw)
        dxs = fb.fp8_moe_gemm_dgrad(qg, sg, self.q1, self.s1, offsets, **kw)
        qxT, sxT = fb.fp8_requantize_colgroup(qx, sx, used=used, **kw)
        dw1 = fb.fp8_moe_gemm_wgrad(qgT, sgT, qxT, sxT, offsets, out_dtype=torch.float32, **kw)
        dx = fb.fp8_moe_combine(dxs, rows, stream=stream)
        dlogits = fb.fp8_moe_route_backward(logits, ids, dweights, renormalize=self.renormalize, stream=stream)
        return y, dx, dlogits, dw1, dw2

    def reference(self, ids):
        """The same in 64 bits, nothing quantized: autograd of the formulas."""
        import torch
        t = lambda b: torch.from_numpy(f64(b)).requires_grad_()  # noqa: E731
        x, logits = t(self.x), t(self.logits)
        w1, w2 = t(self.w1), t(self.w2)
        ids = torch.from_numpy(ids).long()
        live = ids >= 0
        # (a row without any expert has no softmax: masked apart, so that no NaN reaches the gradient)
        some = live.any(1)
        chosen = torch.gather(logits[some], 1, ids[some].clamp(min=0)).masked_fill(~live[some], -np.inf)
        over = chosen if self.renormalize else logits[some]
        p = torch.exp(chosen - torch.logsumexp(over, 1, keepdim=True))
        w = torch.zeros(ids.shape, dtype=torch.float64).masked_scatter(some[:, None].expand(ids.shape), p)
        y = torch.zeros(self.T, self.H, dtype=torch.float64)
        for e in range(self.E):
            tok, i = torch.nonzero(ids == e, as_tuple=True)
            gu = x[tok] @ w1[e * 2 * self.I:(e + 1) * 2 * self.I].T
            h = torch.nn.functional.silu(gu[:, :self.I]) * gu[:, self.I:]
            z = h @ w2[e * self.H:(e + 1) * self.H].T
            y = y.index_add(0, tok, w[tok, i][:, None] * z)
        y.backward(torch.from_numpy(f64(self.dy)))
        return [a.detach().numpy() for a in (y, x.grad, logits.grad, w1.grad, w2.grad)]


# How far quantization may take the step from the unquantized one, as a share of
# a result's norm.  An E4M3 code is off by at most 2^-4 of its value, 2^-4 / sqrt 3
# = 0.036 at most in the mean square, independently from code to code, so each
# quantized operand adds 0.036 of the norm of a product, in quadrature (sums of
# values of random signs do not amplify it).  Into dx and dw1 go dz, w2, and g and u
# (x, w1 and their checkpoint each), (dg, du) and x or w1: ten.  The derivatives of
# silu stay below 1.1 in size, of which the second one scales g's share.  sqrt(10) *
# 0.036 * 1.1 = 0.13; twice that for dlogits, whose sums cancel (a chosen expert's
# value minus the mean of them).  A segment taken for its neighbour, a term left out
# or a transposed operand is off by more than 0.3.
SHARE = {"y": 0.13, "dx": 0.13, "dlogits": 0.26, "dw1": 0.13, "dw2": 0.13}


@MODES
@pytest.mark.parametrize("T,H,I,E,k,renormalize", [(300, 512, 256, 6, 2, True), (1, 128, 128, 3, 2, True),
                                                   (777, 256, 384, 10, 4, False), (129, 384, 640, 1, 1, False)])
def test_step_against_64_bits(T, H, I, E, k, renormalize, mode):
    c = Layer(T, H, I, E, k, mode, 1, renormalize)
    if T == 1:
        c.logits[:] = 0x3F80
    x, logits, dy = c.device()
    got = [host(t) for t in c.step(x, logits, dy)]
    ids = host(fb.fp8_moe_route(logits, k, renormalize=renormalize)[0])
    got = [f64(g) if g.dtype == np.uint16 else g.astype(np.float64) for g in got]
    for name, g, w in zip(SHARE, got, c.reference(ids)):
        w = w.reshape(g.shape)
        assert np.isfinite(g).all(), name
        # one expert of one: its softmax is 1 whatever the logits are, and their gradient 0 but for roundings
        if name == "dlogits" and E == 1:
            assert np.all(np.abs(g) <= 1e-6)
            continue
        if name == "dlogits" and T == 1:     # a single difference of two values, which may cancel
            continue
        assert np.linalg.norm(g - w) <= SHARE[name] * np.linalg.norm(w), name
        rest = np.abs(w).reshape(w.shape[0], -1).sum(1) == 0
        assert (g.reshape(w.shape[0], -1)[rest] == 0).all(), (name, "what has no choice has zeros")


@MODES
def test_step_in_graphs(mode):
    """Two layers' steps captured once each and replayed in turn, with other work and other batches between the replays:
    each replay has the bits of an eager call on what the inputs hold then."""
    import torch
    layers = [Layer(300, 512, 256, 6, 2, mode, 2), Layer(1100, 256, 128, 9, 4, mode, 3)]
    graphs = []
    for c in layers:
        held = c.device()
        c.step(*held)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.step(*held)
        graphs.append((c, held, g, out))
    other = torch.randn(256, 256, device="cuda")
    for i in range(4):
        for c, held, g, out in graphs:
            c.batch(10 + i)
            for h, n in zip(held, c.device()):
                h.copy_(n)
            for o in out:
                o.fill_(3.0)
            other = other @ other.T.contiguous() / 256
            g.replay()
            torch.cuda.synchronize()
            for name, o, w in zip(SHARE, out, c.step(*held)):
                assert torch.equal(o, w), (i, name)


@MODES
def test_step_on_two_streams_at_once(mode):
    """On streams of their own, both layers under way at once: the bits of one after the other."""
    import torch
    layers = [Layer(300, 512, 256, 6, 2, mode, 4), Layer(2100, 256, 128, 40, 4, mode, 5)]
    inputs = [c.device() for c in layers]
    want = [c.step(*i) for c, i in zip(layers, inputs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for explicit in (True, False):
        got = []
        for _ in range(3):
            for c, i, s in zip(layers, inputs, streams):
                if explicit:
                    got.append(c.step(*i, stream=s))
                else:
                    with torch.cuda.stream(s):
                        got.append(c.step(*i))
        torch.cuda.synchronize()
        for n, g in enumerate(got):
            for name, a, b in zip(SHARE, g, want[n % 2]):
                assert torch.equal(a, b), (n, name)


def test_forward_against_the_layer_of_few_tokens():
    """The same layer from the same codes by fp8_moe_experts, which keeps gate, up and the experts' results in fp32."""
    import torch
    c = Layer(64, 512, 256, 6, 2, POW2, 6)
    x, logits, dy = c.device()
    ids, w = fb.fp8_moe_route(logits, 2)
    y = fb.fp8_moe_experts(x, ids, w, c.q1, c.s1, c.q2, c.s2, out_dtype=torch.float32)
    got = c.step(x, logits, dy)[0].float()
    # gate and up, rounded to bf16 (2^-9 each), and h, rounded from there, take h by at most 3 2^-9 = 2^-7.4 from the
    # other's, which moves at most one code in eight to its neighbour (a step is 2^-4 to 2^-3 of the value), by 2^-3.5 on
    # the mean: 2^-3.5 / sqrt(8) = 0.03 of h's norm; the results' own rounding and the sums' order are small beside it
    assert float((got - y).norm()) <= 0.04 * float(y.norm())
    assert bool((got[host(ids)[:, 0] < 0] == 0).all())


def test_two_graphs_share_workspaces():
    """The workspaces of the sort and of a gather in the order of tokens, between two graphs, filled with other bytes
    before each replay."""
    import torch
    sizes = [(12000, 20, 8, 1152), (9001, 40, 8, 1408)]
    need = [(fb.fp8_moe_sort_workspace_size(T, E, k),
             fb.fp8_moe_gather_workspace_size(T, H, fb.fp8_moe_sorted_rows(T, E, k), k)) for T, E, k, H in sizes]
    assert all(n > 0 for pair in need for n in pair)
    ws = [torch.empty(max(p[i] for p in need), dtype=torch.uint8, device="cuda") for i in (0, 1)]
    graphs = []
    for T, E, k, H in sizes:
        gen = torch.Generator("cuda").manual_seed(T)
        ids = torch.randint(-1, E + 1, (T, k), generator=gen, device="cuda").int()
        x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()

        def run(ids=ids, x=x, E=E, k=k):
            rows, source, offsets = fb.fp8_moe_sort(ids, E, workspace=ws[0])
            return rows, source, offsets, *fb.fp8_moe_gather(x, source, k, used=offsets[-1:], workspace=ws[1])

        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out, want, run))
    for _ in range(3):
        for g, out, want, _ in graphs:
            for w in ws:
                w.fill_(0xFF)
            for o in out:
                o.fill_(1)
            g.replay()
            torch.cuda.synchronize()
            used = int(want[2][-1])
            for i, (o, w) in enumerate(zip(out, want)):
                assert torch.equal(o[:used], w[:used]) if i > 2 else torch.equal(o, w), i
