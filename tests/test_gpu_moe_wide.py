"""The mixture's kernels for dozens of rows an expert, each instance of them
(test_moe_paths.py holds the sizes to that), and the narrow gate/up whose
workgroups take several columns; experts with from none to 80 rows."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import moe_cases
import moe_ref
from gpu_util import dev, dev_bf16, host, require_gpu
from test_gpu_moe import _case, _exact_case

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
CASES = moe_cases.WIDE + moe_cases.NARROW


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _ids(T, E, k):
    return moe_cases.uneven_ids(T, E, k, T) if T > 16 else None


@pytest.mark.parametrize("T,H,I,E,k", CASES)
def test_exact(T, H, I, E, k):
    """Whole numbers throughout: no rounding on the way, and the result equal."""
    import torch
    ids = _ids(T, E, k)
    args, _ = _exact_case(T, E, k, 1000 + T, H, I, ids=None if ids is None else np.maximum(ids, 0))
    # (the reference runs over every place; those without an expert weigh nothing there)
    x, w = args[0], args[2].clone()
    chosen = args[1] if ids is None else dev(ids)
    w[chosen < 0] = 0
    ref = _reference(x, chosen.clamp(min=0), w, args)
    y = fb.fp8_moe_experts(x, chosen, args[2], *args[3:], out_dtype=torch.float32)
    assert np.array_equal(host(y).astype(np.float64), ref)
    assert torch.equal(fb.fp8_moe_experts(x, chosen, args[2], *args[3:]), y.bfloat16())
    assert torch.equal(fb.fp8_moe_experts(x, chosen, args[2], *args[3:], out_dtype=torch.float32), y)


def _reference(x, ids, w, args):
    """64-bit result of a whole-number case from its operands as they are on the GPU."""
    xh, ids, w = host(x.float()).astype(np.float64), host(ids), host(w).astype(np.float64)
    w1, w2 = (moe_ref.dequant_block(host(q), host(s)) for q, s in (args[3:5], args[5:7]))
    I = w2.shape[2]
    y = np.zeros_like(xh)
    for e in np.unique(ids):
        t, j = np.nonzero((ids == e) & (w != 0))
        gu = xh[t] @ w1[e].T
        np.add.at(y, t, w[t, j][:, None] * ((gu[:, :I] * gu[:, I:]) @ w2[e].T))  # silu(32) = 32 and silu(64) = 64
    return y


@pytest.mark.parametrize("T,H,I,E,k", CASES)
@pytest.mark.parametrize("mode", [POW2, FP32])
def test_bounded(T, H, I, E, k, mode):
    import torch
    x, ids, w, q1, s1, q2, s2 = _case(T, H, I, E, k, 700 + T, mode, ids=_ids(T, E, k))
    ref, bound = moe_ref.experts(x, ids, w, q1, s1, q2, s2, mode)
    y = fb.fp8_moe_experts(dev_bf16(x), dev(ids), dev(w), dev(q1), dev(s1), dev(q2), dev(s2), out_dtype=torch.float32,
                           scale_mode=mode)
    err = np.abs(host(y).astype(np.float64) - ref)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))
