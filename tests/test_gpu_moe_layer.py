"""fp8_moe_layer where its dispatch changes: tokens that are not finite, every
size of router, both scale rules, experts whose logits tie."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import moe_ref
from blockwise_fp8_linear_amd import synth
from gpu_util import dev, dev_bf16, host, require_gpu
from test_gpu_moe import _case

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _layer(x, wr, exps, k, **kw):
    """(y fp32, ids, weights) of a layer; the buffers hold other values before."""
    import torch
    ids = torch.full((x.shape[0], k), 7, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], k), 7.0, device="cuda")
    return fb.fp8_moe_layer(x, wr, *exps, k, out_dtype=torch.float32, ids=ids, weights=w, **kw), ids, w


# the narrow kernels with the router inside (T 2) and with its logits apart (T 4, 7), several workgroups a column
# (I 8448), the wide gate/up with the narrow down projection (T 14), the wide kernels (T 30)
NOT_FINITE = [(2, 256, 128, 8, 2), (4, 1024, 128, 70, 5), (7, 1024, 128, 70, 3), (3, 256, 8448, 3, 2),
              (14, 128, 512, 64, 8), (14, 1152, 128, 64, 8), (30, 256, 128, 8, 2), (30, 1152, 128, 64, 2)]


@pytest.mark.parametrize("T,H,I,E,k", NOT_FINITE)
@pytest.mark.parametrize("mode", [POW2, FP32])
def test_layer_shows_a_token_that_is_not_finite(T, H, I, E, k, mode):
    """No expert can be chosen for a token whose logits are all NaN (one NaN in
    its row) or all -infinity: its result is NaN, not the zeros of a padded
    token, and the others are as right as before."""
    import torch
    xb, _, _, q1, s1, q2, s2 = _case(T, H, I, E, 1, 600 + T, mode)
    x, exps = dev_bf16(xb), tuple(dev(a) for a in (q1, s1, q2, s2))
    wr = -dev_bf16(synth.normal_bf16((E, H), 0.3, 90, T)).abs() - 0.01
    clean, cids, cw = _layer(x, wr, exps, k, scale_mode=mode)
    # (the narrow down projection adds the blocks of all experts that the call reaches in one order, cut into the waves'
    # parts: without the bad token's experts the others' sums may be cut elsewhere, so they are held to the bound that
    # every order keeps)
    ref, bound = moe_ref.experts(xb, host(cids), host(cw), q1, s1, q2, s2, mode)
    keep = [t for t in range(T) if t != 1]
    for bad in (float("nan"), float("inf")):     # times the negative weights: every logit NaN, every one -infinity
        z = x.clone()
        z[1, H - 3] = bad
        y, ids, w = _layer(z, wr, exps, k, scale_mode=mode)
        assert bool((ids[1] == -1).all()) and bool((w[1] == 0).all())
        assert bool(torch.isnan(y[1]).all())
        assert torch.equal(ids[keep], cids[keep]) and torch.equal(w[keep], cw[keep])
        assert np.all(np.abs(host(y).astype(np.float64) - ref)[keep] <= bound[keep])
        b = fb.fp8_moe_layer(z, wr, *exps, k, scale_mode=mode)
        assert bool(torch.isnan(b[1]).all()) and torch.equal(b[keep], y[keep].bfloat16())
        # the same choice from the caller is a padded token: zeros
        assert bool((fb.fp8_moe_experts(z, ids, w, *exps, scale_mode=mode)[1] == 0).all())
    z = x.clone()
    z[1] = 0                                     # a row of zeros ties all experts and is a row of zeros again
    y, ids, _ = _layer(z, wr, exps, k, scale_mode=mode)
    assert host(ids[1]).tolist() == list(range(k)) and bool((y[1] == 0).all())
    assert bool(torch.isfinite(clean).all())


# routers of every size class: inside the token's own launch (E H <= 64 Ki; 2 to 8 rounds of 64 experts), in the narrow
# gate/up with 4, 8 and 16 tokens' rows, and in the wide kernels' token launch
ROUTERS = [(5, 128, 128, 129, 4), (30, 128, 128, 257, 3), (3, 128, 128, 512, 16), (40, 128, 128, 512, 2),
           (1, 128, 128, 1024, 16), (3, 128, 128, 1024, 5), (6, 512, 128, 200, 5), (12, 512, 128, 200, 3),
           (12, 128, 128, 1024, 2), (20, 128, 128, 1024, 16), (17, 640, 128, 256, 7)]


@pytest.mark.parametrize("T,H,I,E,k", ROUTERS)
@pytest.mark.parametrize("mode", [POW2, FP32])
def test_layer_chooses_and_ties(T, H, I, E, k, mode):
    """Each expert of the first half stands again in the second, with the same
    logit: the lower index comes first.  The choice is held to 64-bit logits (an
    fp32 sum may exchange what lies closer than its error), the weights to the
    softmax of the choice, the result to the experts' own call."""
    import torch
    x, _, _, q1, s1, q2, s2 = _case(T, H, I, E, 1, 800 + T, mode)
    wr = synth.normal_bf16((E, H), 0.3, 94, T + E)
    half = E // 2
    wr[half:2 * half] = wr[:half]
    exps, renorm = tuple(dev(a) for a in (q1, s1, q2, s2)), T % 2 == 0
    y, ids, w = _layer(dev_bf16(x), dev_bf16(wr), exps, k, renormalize=renorm, scale_mode=mode)
    lg = moe_ref.f64(x) @ moe_ref.f64(wr).T
    err = (H + 16) * 2 * moe_ref.U * (np.abs(moe_ref.f64(x)) @ np.abs(moe_ref.f64(wr)).T).max()
    got, gw = host(ids), host(w).astype(np.float64)
    for t in range(T):
        row, chosen = lg[t], list(got[t])
        assert len(set(chosen)) == k and 0 <= min(chosen) and max(chosen) < E
        assert np.all(np.abs(row[chosen] - np.sort(row)[::-1][:k]) <= 2 * err)
        for at, e in enumerate(chosen):
            if half <= e < 2 * half:
                assert e - half in chosen[:at], (t, chosen)
        p = moe_ref._softmax(row, chosen if renorm else list(range(E)))
        rw = np.array([p[j] for j in chosen])
        assert np.all(np.abs(gw[t] - rw) <= (2 * err + moe_ref.route_tolerance(np.ptp(row), E)) * 1.01 * rw)
    assert torch.equal(y, fb.fp8_moe_experts(dev_bf16(x), ids, w, *exps, out_dtype=torch.float32, scale_mode=mode))
    b = fb.fp8_moe_layer(dev_bf16(x), dev_bf16(wr), *exps, k, renormalize=renorm, scale_mode=mode)
    assert torch.equal(b, y.bfloat16())
