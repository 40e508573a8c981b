"""The experts' products on every kind of tile, on the GPU: output types, results
that do not depend on the other experts, offsets that are no whole blocks, are
outside the buffer or descend."""
import numpy as np
import pytest

import blockwise_fp8_linear_amd as fb
import expert_cases
from gpu_util import RTOL, require_gpu

pytestmark = pytest.mark.gpu

POW2, FP32 = fb.FP8BLK_SCALE_POW2, fb.FP8BLK_SCALE_FP32
MODES = pytest.mark.parametrize("mode", [POW2, FP32])
SIZES = pytest.mark.parametrize("size", [size for size, _ in expert_cases.SIZES], ids=lambda s: "-".join(map(str, s)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _release():
    yield
    import torch
    torch.cuda.empty_cache()


class Experts:
    """Operands of one product for segments of `lengths` rows: an expert's rows are the same ones wherever they stand."""

    def __init__(self, size, mode, key):
        import torch
        self.way, self.N, self.K, self.E, self.R = size
        self.mode = mode
        self.g = torch.Generator("cuda").manual_seed(key)
        self.x = [self.normal(self.R, c) for c in ((self.N, self.K) if self.way == "wgrad" else (self.red,))]
        if self.way != "wgrad":
            qw, _, sw = fb.fp8_quantize_block(self.normal(self.E * self.N, self.K, 0.02), transpose=False, scale_mode=mode)
            self.w = qw.view(self.E, self.N, self.K), sw.view(self.E, self.N // 128, self.K // 128)

    @property
    def red(self):
        return self.K if self.way == "fprop" else self.N

    @property
    def shape(self):
        return {"fprop": (self.R, self.N), "dgrad": (self.R, self.K), "wgrad": (self.E, self.N, self.K)}[self.way]

    def normal(self, rows, cols, std=1.0):
        import torch
        x = torch.randn((rows, cols), generator=self.g, device="cuda") * std
        return (x * torch.randint(-3, 4, (rows, 1), generator=self.g, device="cuda").float().exp2()).bfloat16()

    def place(self, lengths, fixed=None):
        """Quantize rows in these segments; those of expert `fixed` are the first ones there are, the others' are others."""
        import torch
        self.offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        order = torch.roll(torch.arange(self.R, device="cuda"), 128 * 3 + 128)
        if fixed is not None:
            lo, hi = int(self.offsets[fixed]), int(self.offsets[fixed + 1])
            first = torch.arange(hi - lo, device="cuda")
            others = torch.arange(hi - lo, self.R, device="cuda")
            order = torch.cat([others[:lo], first, others[lo:]])
        if self.way == "wgrad":
            self.a, self.b = (fb.fp8_quantize_colgroup(x[order].contiguous(), scale_mode=self.mode) for x in self.x)
        else:
            self.a, self.b = fb.fp8_quantize_rowgroup(self.x[0][order].contiguous(), scale_mode=self.mode), self.w

    def run(self, offsets=None, **kw):
        import torch
        f = {"fprop": fb.fp8_moe_gemm_fprop, "dgrad": fb.fp8_moe_gemm_dgrad, "wgrad": fb.fp8_moe_gemm_wgrad}[self.way]
        off = torch.from_numpy(self.offsets if offsets is None else np.array(offsets, np.int32)).cuda()
        return f(*self.a, *self.b, off, scale_mode=self.mode, **kw)

    def rows_in_use(self, out):
        return out if self.way == "wgrad" else out[:int(self.offsets[-1])]

    def want(self):
        """(the result in 64 bits, the sums of magnitudes), of the rows in use."""
        import torch

        def value(q, s, block=False):
            s = s.double().repeat_interleave(128, 1)
            return q.view(torch.float8_e4m3fn).double() * (s.repeat_interleave(128, 0) if block else s)

        y, size = (torch.zeros(self.shape, dtype=torch.float64, device="cuda") for _ in range(2))
        for e in range(self.E):
            lo, hi = int(self.offsets[e]), int(self.offsets[e + 1])
            if lo == hi:
                continue
            if self.way == "wgrad":
                a, b = (value(q[:, lo:hi], s[:, lo // 128:hi // 128]) for q, s in (self.a, self.b))
                b, at = b.T.contiguous(), e
            else:
                a = value(self.a[0][lo:hi], self.a[1][lo:hi])
                b = value(self.b[0][e], self.b[1][e], True)
                b, at = b.T.contiguous() if self.way == "fprop" else b, slice(lo, hi)
            y[at], size[at] = a @ b, a.abs() @ b.abs()
        return self.rows_in_use(y), self.rows_in_use(size)


@MODES
@SIZES
@pytest.mark.parametrize("which", [0, 1, 3])
def test_types(size, which, mode):
    """fp32 against 64 bits; bf16, and what is added to, have the fp32 result; rows of no segment stay."""
    import torch
    c = Experts(size, mode, 31)
    c.place(expert_cases.spreads(c.E, c.R)[1][which])
    room = torch.full((c.shape[0] + 2, *c.shape[1:]), -0.5, device="cuda")
    out = room[1:-1]
    c.run(out_dtype=torch.float32, out=out)
    y, sums = c.want()
    err = (c.rows_in_use(out) - y).abs()
    assert bool((err <= RTOL * sums).all())     # 0 where there is nothing to add
    # the instruction's sums are off by 1.5e-5 .. 4.5e-5 of the result's norm; a term left out by 1 / sqrt(5120) or more
    assert float(err.norm()) <= 2e-4 * float(y.norm())
    used = room.shape[0] - 1 if c.way == "wgrad" else 1 + int(c.offsets[-1])
    assert bool((room[0] == -0.5).all()) and bool((room[used:] == -0.5).all())
    b = torch.full_like(room, -0.5, dtype=torch.bfloat16)
    c.run(out=b[1:-1])
    assert torch.equal(b, room.bfloat16())
    acc = torch.randn(room.shape, generator=c.g, device="cuda")
    want = acc.clone()
    want[1:used] += room[1:used]
    c.run(out_dtype=torch.float32, out=acc[1:-1], accumulate=True)
    assert torch.equal(acc, want)


@MODES
@SIZES
def test_results_do_not_depend_on_the_other_experts(size, mode):
    """An expert's rows, bit for bit, among four spreads of the rest over the others, at the same sizes."""
    import torch
    c = Experts(size, mode, 32)
    e, lists = expert_cases.spreads(c.E, c.R)
    seen = []
    for lengths in lists:
        c.place(lengths, fixed=e)
        out = c.run(out_dtype=torch.float32)
        lo, hi = int(c.offsets[e]), int(c.offsets[e + 1])
        seen.append(out[e] if c.way == "wgrad" else out[lo:hi])
        assert torch.equal(c.run(out_dtype=torch.float32)[e if c.way == "wgrad" else slice(lo, hi)], seen[-1])
    assert bool(seen[0].abs().max() > 0) and all(torch.equal(s, seen[0]) for s in seen[1:])


@MODES
@SIZES
def test_odd_offsets_stay_inside(size, mode):
    """Offsets outside the buffer or between multiples of 128 count as documented; descending ones touch nothing else."""
    import torch
    c = Experts(size, mode, 33)
    lengths = expert_cases.spreads(c.E, c.R)[1][1]
    lengths[-1] = c.R - sum(lengths[:-1])       # up to the end
    c.place(lengths)
    ok = c.run(out_dtype=torch.float32)
    odd = c.offsets + np.arange(c.E + 1) * 5 % 128
    odd[0], odd[-1] = -300, 2 ** 31 - 1
    assert torch.equal(c.run(odd, out_dtype=torch.float32), ok)
    room = torch.full((c.shape[0] + 2, *c.shape[1:]), -0.5, device="cuda")
    down = c.offsets.copy()
    down[2], down[3], down[c.E - 2] = c.R, 128, -2 ** 31
    c.run(down, out_dtype=torch.float32, out=room[1:-1])
    c.run(down[::-1].copy(), out_dtype=torch.float32, out=room[1:-1])
    assert bool((room[0] == -0.5).all()) and bool((room[-1] == -0.5).all())


@MODES
@pytest.mark.parametrize("size", [size for size, _ in expert_cases.SIZES if size[0] == "wgrad"],
                         ids=lambda s: "-".join(map(str, s)))
def test_accumulating_nothing_leaves_every_bit(size, mode):
    """An expert without rows keeps what was there, negative zeros and NaN among it."""
    import torch
    c = Experts(size, mode, 34)
    e, lists = expert_cases.spreads(c.E, c.R)
    c.place(lists[0])       # that expert alone has rows
    was = torch.randint(-2 ** 31, 2 ** 31 - 1, c.shape, generator=c.g, device="cuda", dtype=torch.int32)
    was[:, :, ::5] = -2 ** 31
    out = was.clone().view(torch.float32)
    c.run(out_dtype=torch.float32, out=out, accumulate=True)
    for i in range(c.E):
        assert torch.equal(out[i].view(torch.int32), was[i]) == (i != e), i
