"""include/fp8moe.h and its binding, checked without a GPU: the library
exports what the header declares, every argument error has its documented
status before anything is launched (the pointers are never dereferenced), the
limits and workspace sizes are consistent, the header is C, and the binding
refuses operands that disagree with the sizes it would pass."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import blockwise_fp8_linear_amd as fb
from blockwise_fp8_linear_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ENULL, EDIM, EALIGN, EARG, EWS, EHIP, EDEV = 0, -1, -2, -3, -4, -5, -6, -7
NOGPU = (EHIP, EDEV)      # what valid arguments give on a machine without a gfx950
BAD = ctypes.c_size_t(-1).value
P = [0x100000 * i for i in range(1, 12)]    # fake aligned addresses


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: valid arguments would launch on fake addresses")
    return moe._functions()


def caller(f, names, good):
    def call(**kw):
        assert set(kw) <= set(names)
        a = dict(zip(names, good))
        a.update(kw)
        return f(*[a[n] for n in names])
    return call


def test_exports_every_declared_function():
    names = set(fb.header_functions(moe.HEADER_PATH))
    assert names == {"fp8_linear", "fp8_linear_workspace_size", "fp8_moe_route", "fp8_moe_route_backward",
                     "fp8_moe_experts", "fp8_moe_layer", "fp8_moe_workspace_size"}
    lib = moe._functions()
    for n in names:
        assert hasattr(lib, n) and callable(getattr(fb, n)), n


def test_constants_are_the_headers():
    text = open(moe.HEADER_PATH).read()
    for n in ("FP8_LINEAR_FP32_ROWS", "FP8MOE_MAX_EXPERTS", "FP8MOE_MAX_TOPK", "FP8MOE_MAX_TOKENS"):
        assert int(re.search(rf"#define {n} (\d+)", text).group(1)) == getattr(fb, n)
    for n in ("FP8MOE_BF16", "FP8MOE_FP32"):
        assert int(re.search(rf"{n} = (\d+)", text).group(1)) == getattr(fb, n)


def test_linear_errors(lib):
    names = ("M", "N", "K", "x", "ld", "qw", "sw", "y", "odt", "mode", "ws", "wsb", "stream")
    call = caller(lib.fp8_linear, names, (3, 256, 384, P[0], 384, P[1], P[2], P[3], 0, 0, None, 0, None))
    assert call() in NOGPU
    for odt in (1, 2):
        assert call(odt=odt) in NOGPU
    assert call(mode=1) in NOGPU
    for kw in ({"odt": 3}, {"odt": -1}, {"mode": 2}, {"mode": -1}, {"ld": 256}, {"ld": 1 << 27},
               {"K": 128 << 18, "ld": 128 << 18}, {"M": 1 << 27}, {"N": 1 << 30, "M": 1 << 20}):
        assert call(**kw) == EARG, kw
    for n in ("x", "qw", "sw", "y"):
        assert call(**{n: None}) == ENULL, n
    for kw in ({"M": 0}, {"M": -1}, {"N": 0}, {"N": 200}, {"K": 0}, {"K": 100, "ld": 104}):
        assert call(**kw) == EDIM, kw
    for kw in ({"x": P[0] + 8}, {"qw": P[1] + 8}, {"y": P[3] + 4}, {"sw": P[2] + 2}, {"ld": 388}):
        assert call(**kw) == EALIGN, kw
    for mode in (0, 1):
        need = lib.fp8_linear_workspace_size(300, 4096, 2048, mode)
        assert need >= 300 * 2048 + 300 * 16 * 4
        big = {"M": 300, "N": 4096, "K": 2048, "ld": 2048, "mode": mode}
        assert call(**big) == EWS and call(**big, ws=P[4], wsb=need - 1) == EWS
        assert call(**big, ws=P[4] + 8, wsb=need) == EALIGN
        assert call(**big, ws=P[4], wsb=need) in NOGPU


def test_linear_workspace(lib):
    q = lib.fp8_linear_workspace_size
    assert q(1, 128, 128, 0) == 0 and q(8, 12288, 2048, 1) == 0 and q(300, 256, 384, 0) == 0
    assert q(40, 12288, 2048, 0) == 0 and q(40, 12288, 2048, 1) > 0
    assert q(1, 128, 128, 2) == BAD and q(1, 128, 128, -1) == BAD
    for bad in ((0, 128, 128), (1, 100, 128), (1, 128, 100), (1 << 27, 128, 128), (1, 128, 128 << 18),
                (1 << 62, 128, 128)):
        assert q(*bad, 0) == BAD, bad
    # codes and scales of every row that is quantized first, whichever kernel takes it
    for M, N, K, few in ((64, 12288, 2048, 0), (127, 4096, 4096, 0), (333, 2048, 2048, 0), (4133, 4096, 2048, 37),
                         (1100, 8192, 2048, 76)):
        for mode in (0, 1):
            assert q(M, N, K, mode) >= (M - few) * (K + K // 128 * 4)


def test_route_errors(lib):
    names = ("T", "E", "k", "lg", "dt", "ld", "re", "ids", "w", "stream")
    call = caller(lib.fp8_moe_route, names, (3, 10, 2, P[0], 0, 10, 1, P[1], P[2], None))
    assert call() in NOGPU and call(dt=1, re=0, ld=17) in NOGPU and call(E=1024, ld=1024, k=16) in NOGPU
    for kw in ({"dt": 2}, {"re": 2}, {"ld": 9}, {"E": 1025, "ld": 2000}, {"k": 17, "E": 64, "ld": 64}, {"k": 11},
               {"T": 1 << 31}, {"ld": 1 << 50}):
        assert call(**kw) == EARG, kw
    for n in ("lg", "ids", "w"):
        assert call(**{n: None}) == ENULL, n
    for kw in ({"T": 0}, {"E": 0}, {"k": 0}, {"k": -3}):
        assert call(**kw) == EDIM, kw
    for kw in ({"lg": P[0] + 1}, {"lg": P[0] + 2, "dt": 1}, {"ids": P[1] + 2}, {"w": P[2] + 1}):
        assert call(**kw) == EALIGN, kw
    names = ("T", "E", "k", "lg", "dt", "ld", "ids", "g", "re", "d", "ldd", "stream")
    call = caller(lib.fp8_moe_route_backward, names, (3, 10, 2, P[0], 1, 10, P[1], P[2], 0, P[3], 10, None))
    assert call() in NOGPU and call(ldd=12) in NOGPU
    for kw in ({"ldd": 9}, {"dt": 7}, {"k": 11}, {"ldd": 1 << 50}):
        assert call(**kw) == EARG, kw
    for n in ("lg", "ids", "g", "d"):
        assert call(**{n: None}) == ENULL, n
    assert call(T=0) == EDIM and call(d=P[3] + 2) == EALIGN


LAYER = ("T", "H", "I", "E", "k", "re", "x", "ld", "wr", "q1", "s1", "q2", "s2", "y", "odt", "mode", "ids", "w", "ws",
         "wsb", "stream")


def test_moe_errors(lib):
    need = lib.fp8_moe_workspace_size(5, 256, 128, 8, 2)
    assert 0 < need < BAD
    good = (5, 256, 128, 8, 2, 1, P[0], 256, P[1], P[2], P[3], P[4], P[5], P[6], 0, 0, None, None, P[7], need, None)
    call = caller(lib.fp8_moe_layer, LAYER, good)
    assert call() in NOGPU and call(odt=1, mode=1, re=0, ids=P[8], w=P[9], ld=264) in NOGPU
    for kw in ({"odt": 2}, {"odt": 5}, {"mode": 3}, {"re": -1}, {"T": 513}, {"E": 1025}, {"k": 9}, {"E": 64, "k": 17},
               {"ld": 248}, {"ld": 1 << 27}, {"H": 1 << 21, "ld": 1 << 21}, {"I": 1 << 21},
               {"H": 1 << 20, "I": 1 << 20, "ld": 1 << 20}, {"T": 512, "E": 64, "k": 16, "I": 1 << 18}):
        assert call(**kw) == EARG, kw
    for n in ("x", "wr", "q1", "s1", "q2", "s2", "y"):
        assert call(**{n: None}) == ENULL, n
    for kw in ({"T": 0}, {"H": 0}, {"H": 200, "ld": 200}, {"I": 64}, {"E": 0}, {"k": 0}):
        assert call(**kw) == EDIM, kw
    for kw in ({"x": P[0] + 8}, {"wr": P[1] + 2}, {"q1": P[2] + 4}, {"q2": P[4] + 8}, {"y": P[6] + 8}, {"s1": P[3] + 2},
               {"s2": P[5] + 1}, {"ids": P[8] + 2}, {"w": P[9] + 2}, {"ld": 260}, {"ws": P[7] + 4}):
        assert call(**kw) == EALIGN, kw
    assert call(ws=None) == EWS and call(wsb=need - 1) == EWS
    names = ("T", "H", "I", "E", "k", "x", "ld", "ids", "w", "q1", "s1", "q2", "s2", "y", "odt", "mode", "ws", "wsb",
             "stream")
    call = caller(lib.fp8_moe_experts, names, (5, 256, 128, 8, 2, P[0], 256, P[8], P[9], P[2], P[3], P[4], P[5], P[6], 0,
                                               0, P[7], need, None))
    assert call() in NOGPU
    for n in ("x", "ids", "w", "q1", "y"):
        assert call(**{n: None}) == ENULL, n
    assert call(T=513) == EARG and call(I=100) == EDIM and call(ws=None) == EWS


def test_moe_workspace(lib):
    q = lib.fp8_moe_workspace_size
    for bad in ((0, 128, 128, 1, 1), (1, 100, 128, 1, 1), (1, 128, 100, 1, 1), (513, 128, 128, 1, 1),
                (1, 128, 128, 1025, 1), (1, 128, 128, 4, 5), (1, 128, 128, 4, 0), (1, 1 << 62, 128, 4, 1)):
        assert q(*bad) == BAD, bad
    for T, H, I, E, k in ((1, 128, 128, 1, 1), (16, 2048, 1024, 64, 16), (17, 2048, 6144, 8, 2), (512, 256, 128, 1024, 16)):
        # logits, choice, x's codes and scales, h, its scales, partial results (16 workgroups a column at most, few tokens)
        least = T * E * 4 + T * k * 8 + T * H + T * (H // 128) * 4 + T * k * I * 2 + T * k * (I // 128) * 4
        assert q(T, H, I, E, k) >= least + (max(k, 16) if T <= 16 else k) * T * H * 4


def test_host_checks_under_sanitizers(tmp_path):
    """api_moe.cpp under gcc's address and undefined-behaviour sanitizers, its
    launchers replaced by stubs that record where each would read and write."""
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no g++ or no HIP headers")
    csrc, exe = os.path.join(ROOT, "blockwise_fp8_linear_amd", "csrc"), str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                    "-isystem", "/opt/rocm/include", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "api_moe_host_check.cpp"),
                    os.path.join(csrc, "api_moe.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-4000:] + r.stderr[-4000:]


def test_header_is_c(tmp_path):
    if shutil.which("gcc") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no gcc or no HIP headers")
    src, exe = tmp_path / "c.c", str(tmp_path / "c")
    src.write_text('#include "fp8moe.h"\n#include <stdio.h>\nint main(void) {\n'
                   "  if (fp8_linear(0, 128, 128, 0, 128, 0, 0, 0, 0, 0, 0, 0, 0) != FP8BLK_ERR_NULL) return 1;\n"
                   "  if (fp8_moe_route(1, 4, 9, 0, FP8MOE_FP32, 4, 1, 0, 0, 0) != FP8BLK_ERR_NULL) return 2;\n"
                   "  if (fp8_moe_route_backward(1, 4, 2, 0, 9, 4, 0, 0, 1, 0, 4, 0) != FP8BLK_ERR_ARG) return 3;\n"
                   "  if (fp8_moe_experts(1, 128, 128, 4, 2, 0, 128, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != FP8BLK_ERR_NULL) "
                   "return 4;\n"
                   "  if (fp8_moe_layer(1, 128, 128, 4, 2, 1, 0, 128, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != "
                   "FP8BLK_ERR_NULL) return 5;\n"
                   "  if (fp8_linear_workspace_size(0, 1, 1, 0) != (size_t)-1) return 6;\n"
                   "  if (fp8_moe_workspace_size(FP8MOE_MAX_TOKENS + 1, 128, 128, 4, 2) != (size_t)-1) return 7;\n"
                   '  puts("ok");\n  return 0;\n}\n')
    libdir = os.path.dirname(fb.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-isystem", "/opt/rocm/include", str(src), "-o", exe, "-L", libdir,
                    "-l:libfp8blk.so", f"-Wl,-rpath,{libdir}"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)


# ------------------------------------------------------------- the binding --

u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


class NoLibrary:
    """Stands in for the library: workspace queries answer, a launch fails the test."""

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 64
        return lambda *a: pytest.fail("the C library was reached with bad operands")


@pytest.fixture
def host_stand_ins(monkeypatch):
    monkeypatch.setattr(moe, "_functions", NoLibrary)
    monkeypatch.setattr(moe, "_linear_need", lambda *a: 64)
    monkeypatch.setattr(moe, "_moe_need", lambda *a: 64)
    monkeypatch.setattr(moe, "_index", lambda x, name: -1 if isinstance(x, torch.Tensor) else pytest.fail(name))
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 0)


def z(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def refused(match, fn, *args, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*args, **kw)


def test_binding_linear(host_stand_ins):
    x, qw, sw = z((5, 256), bf16), z((384, 256), u8), z((3, 2), f32)
    refused("x: expected", fb.fp8_linear, z((5, 256), f32), qw, sw)
    refused("2 dims", fb.fp8_linear, z((5, 2, 256), bf16), qw, sw)
    refused("last dimension", fb.fp8_linear, z((256, 5), bf16).t(), qw, sw)
    refused("qw: expected shape", fb.fp8_linear, x, z((384, 128), u8), sw)
    refused("qw: expected torch.uint8", fb.fp8_linear, x, z((384, 256), torch.int8), sw)
    refused("qw: must be contiguous", fb.fp8_linear, x, z((256, 384), u8).t(), sw)
    refused("sw: expected shape", fb.fp8_linear, x, qw, z((3, 1), f32))
    refused("out: expected shape", fb.fp8_linear, x, qw, sw, out=z((4, 384), bf16))
    refused("out: expected torch.float32", fb.fp8_linear, x, qw, sw, out=z((5, 384), bf16), out_dtype=f32)
    refused("out: must be contiguous", fb.fp8_linear, x, qw, sw, out=z((5, 400), bf16)[:, :384])
    refused("accumulate", fb.fp8_linear, x, qw, sw, accumulate=True)
    refused("out_dtype", fb.fp8_linear, x, qw, sw, out_dtype=torch.float16)
    refused("workspace", fb.fp8_linear, x, qw, sw, workspace=7)
    refused("workspace: must be contiguous", fb.fp8_linear, x, qw, sw, workspace=z((8, 8), f32).t()[1:])


def test_binding_route(host_stand_ins):
    lg = z((5, 9), f32)
    refused("logits: expected", fb.fp8_moe_route, z((5, 9), torch.float16), 2)
    refused("ids: expected shape", fb.fp8_moe_route, lg, 2, ids=z((5, 3), i32))
    refused("ids: expected torch.int32", fb.fp8_moe_route, lg, 2, ids=z((5, 2), torch.int64))
    refused("weights: expected torch.float32", fb.fp8_moe_route, lg, 2, weights=z((5, 2), bf16))
    refused("topk", fb.fp8_moe_route, lg, 2 ** 32 + 2)      # not the 2 that an int would keep of it
    refused("topk", fb.fp8_moe_route_backward, lg, z((5, 1), i32).expand(5, 2 ** 32 + 2), z((5, 1), f32))
    ids, g = z((5, 2), i32), z((5, 2), f32)
    refused("ids: expected a 2-dim", fb.fp8_moe_route_backward, lg, z((10,), i32), g)
    refused("ids: expected shape", fb.fp8_moe_route_backward, lg, z((4, 2), i32), g)
    refused("dweights: expected shape", fb.fp8_moe_route_backward, lg, ids, z((5, 1), f32))
    refused("dlogits: expected torch.float32", fb.fp8_moe_route_backward, lg, ids, g, dlogits=z((5, 9), bf16))
    refused("dlogits: expected shape", fb.fp8_moe_route_backward, lg, ids, g, dlogits=z((5, 8), f32))
    refused("dlogits: the last", fb.fp8_moe_route_backward, lg, ids, g, dlogits=z((9, 5), f32).t())


def test_binding_experts(host_stand_ins):
    T, H, I, E, k = 3, 256, 128, 4, 2
    x, ids, w = z((T, H), bf16), z((T, k), i32), z((T, k), f32)
    good = [z((E, 2 * I, H), u8), z((E, 2 * I // 128, H // 128), f32), z((E, H, I), u8),
            z((E, H // 128, I // 128), f32)]
    wrong = [z((E, 2 * I, H // 2), u8), z((E, 1, 2), f32), z((E, I, H), u8), z((E - 1, 2, 1), f32)]
    for i, name in enumerate(("qw1", "sw1", "qw2", "sw2")):
        e = list(good)
        e[i] = wrong[i]
        refused(f"{name}: expected shape", fb.fp8_moe_experts, x, ids, w, *e)
        refused(f"{name}: expected shape", fb.fp8_moe_layer, x, z((E, H), bf16), *e, k)
    refused("qw1: expected a 3-dim", fb.fp8_moe_experts, x, ids, w, z((E, 3, H), u8), *good[1:])
    refused("ids: expected shape", fb.fp8_moe_experts, x, z((T + 1, k), i32), w, *good)
    refused("weights: expected shape", fb.fp8_moe_experts, x, ids, z((T, k + 1), f32), *good)
    refused("x: expected", fb.fp8_moe_experts, z((T, H), f32), ids, w, *good)
    refused("out: expected shape", fb.fp8_moe_experts, x, ids, w, *good, out=z((T, I), bf16))
    refused("out_dtype", fb.fp8_moe_experts, x, ids, w, *good, out_dtype=torch.float16)
    refused("wr: expected shape", fb.fp8_moe_layer, x, z((E + 1, H), bf16), *good, k)
    refused("wr: expected torch.bfloat16", fb.fp8_moe_layer, x, z((E, H), f32), *good, k)
    refused("ids: expected shape", fb.fp8_moe_layer, x, z((E, H), bf16), *good, k, ids=z((T, k + 1), i32))
    refused("topk", fb.fp8_moe_layer, x, z((E, H), bf16), *good, 2 ** 32 + k)


def test_binding_refuses_host_tensors_and_other_devices():
    """Without stand-ins: a host tensor is no operand, wherever it stands."""
    for fn, args in ((fb.fp8_linear, (z((1, 128), bf16), z((128, 128), u8), z((1, 1), f32))),
                     (fb.fp8_moe_route, (z((1, 4), f32), 2)),
                     (fb.fp8_moe_route_backward, (z((1, 4), f32), z((1, 2), i32), z((1, 2), f32)))):
        refused("device tensor", fn, *args)
    refused("expected a torch.Tensor", fb.fp8_linear, [1.0], None, None)
    with pytest.raises(AttributeError):
        fb.no_such_name
