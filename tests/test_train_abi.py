"""include/fp8train.h and its binding, checked without a GPU: the library exports
what the header declares, every argument error has its documented status before
anything is launched (the pointers are never dereferenced), sizes are consistent,
the header is C, and the binding refuses operands that disagree with the sizes it
would pass."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import blockwise_fp8_linear_amd as fb
import train_ref
from blockwise_fp8_linear_amd import train
from test_moe_abi import BAD, EALIGN, EARG, EDIM, ENULL, EWS, NOGPU, P, ROOT, bf16, caller, f32, i32, refused, u8, z

NAMES = {"fp8_moe_sorted_rows", "fp8_moe_gather_workspace_size", "fp8_moe_sort_workspace_size", "fp8_moe_sort", "fp8_moe_gather", "fp8_moe_combine",
         "fp8_moe_combine_backward", "fp8_moe_gemm_fprop", "fp8_moe_gemm_dgrad", "fp8_moe_gemm_wgrad",
         "fp8_gated_forward", "fp8_gated_backward", "fp8_requantize_colgroup"}
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: valid arguments would launch on fake addresses")
    return train._functions()


def check(call, arg=(), null=(), dim=(), align=(), fine=()):
    assert call() in NOGPU
    for kw in fine:
        assert call(**kw) in NOGPU, kw
    for kw in arg:
        assert call(**kw) == EARG, kw
    for n in null:
        assert call(**{n: None}) == ENULL, n
    for kw in dim:
        assert call(**kw) == EDIM, kw
    for kw in align:
        assert call(**kw) == EALIGN, kw


def test_exports_every_declared_function():
    assert set(fb.header_functions(train.HEADER_PATH)) == NAMES
    lib = train._functions()
    for n in NAMES:
        assert hasattr(lib, n) and callable(getattr(fb, n)), n


def test_sort_errors(lib):
    names = ("T", "E", "k", "ids", "rows", "source", "off", "ws", "wsb", "stream")
    call = caller(lib.fp8_moe_sort, names, (3, 10, 2, P[0], P[1], P[2], P[3], None, 0, None))
    check(call, arg=({"T": 1 << 24}, {"E": 1025}, {"k": 17, "E": 64}, {"k": 11}, {"T": BIG}),
          null=("ids", "rows", "source", "off"), dim=({"T": 0}, {"T": -1}, {"E": 0}, {"k": 0}, {"k": -3}),
          align=tuple({n: P[0] + 2} for n in ("ids", "rows", "source", "off")), fine=({"E": 1024, "k": 16},))
    need = lib.fp8_moe_sort_workspace_size(16384, 128, 8)
    assert need > 0
    big = dict(T=16384, E=128, k=8)
    assert call(**big) == EWS and call(**big, ws=P[4], wsb=need - 1) == EWS
    assert call(**big, ws=P[4] + 4, wsb=need) == EALIGN and call(**big, ws=P[4], wsb=need) in NOGPU


def test_sort_sizes(lib):
    for T, E, k in ((1, 1, 1), (1, 8, 2), (7, 8, 2), (128, 1, 1), (4095, 60, 4), (16384, 128, 8), ((1 << 24) - 1, 1024, 16)):
        assert lib.fp8_moe_sorted_rows(T, E, k) == train_ref.sorted_rows(T, E, k) == fb.fp8_moe_sorted_rows(T, E, k)
    for bad in ((0, 1, 1), (1 << 24, 8, 2), (1, 0, 1), (1, 1025, 1), (4, 4, 5), (4, 64, 17), (4, 4, 0)):
        assert lib.fp8_moe_sorted_rows(*bad) == BAD and lib.fp8_moe_sort_workspace_size(*bad) == BAD, bad
        refused("no such choice", fb.fp8_moe_sorted_rows, *bad)
    assert lib.fp8_moe_sort_workspace_size(7, 8, 2) == 0      # one workgroup counts for itself


GATHER = ("T", "H", "R", "k", "x", "ld", "src", "w", "used", "q", "ldq", "s", "qT", "ldT", "sT", "mode", "ws", "wsb",
          "stream")


def test_gather_errors(lib):
    call = caller(lib.fp8_moe_gather, GATHER, (5, 256, 512, 2, P[0], 256, P[1], None, None, P[2], 256, P[3], P[4], 512,
                                               P[5], 0, None, 0, None))
    check(call, null=("x", "src", "q", "s", "qT", "sT"), fine=({"qT": None, "sT": None, "ldT": 0}, {"w": P[6], "mode": 1},
                                                               {"used": P[7], "ld": 264, "ldq": 272, "ldT": 528}),
          arg=({"mode": 2}, {"k": 17}, {"T": 1 << 24}, {"R": 1 << 31, "ldT": 1 << 31}, {"ld": 248}, {"ldq": 240}, {"ldT": 496},
               {"ld": 1 << 40}, {"ldq": 1 << 40}, {"ldT": 1 << 40}, {"R": 1 << 30, "ldT": 1 << 30}, {"T": BIG},
               {"H": 1 << 30, "ld": 1 << 30, "ldq": 1 << 30},
               {"T": (1 << 24) - 1, "H": 4096, "ld": 4096, "ldq": 4096}),
          dim=({"T": 0}, {"k": 0}, {"H": 0}, {"H": 200}, {"R": 0}, {"R": 100}),
          align=({"x": P[0] + 8}, {"ld": 260}, {"q": P[2] + 4}, {"ldq": 264}, {"s": P[3] + 2}, {"qT": P[4] + 8}, {"ldT": 520},
                 {"sT": P[5] + 1}, {"src": P[1] + 2}, {"w": P[6] + 2}, {"used": P[7] + 1}))


def test_gather_workspace(lib):
    q = lib.fp8_moe_gather_workspace_size
    assert q(5, 256, 512, 2, 0) == q(5, 256, 512, 2, 1) == q(16384, 2048, 139264, 8, 1) == 0
    need = q(16384, 2048, 139264, 8, 0)
    assert need > 0 and fb.fp8_moe_gather_workspace_size(16384, 2048, 139264, 8) == need
    for bad in ((0, 256, 512, 2), (5, 200, 512, 2), (5, 256, 100, 2), (5, 256, 512, 17), (1 << 24, 256, 512, 2)):
        assert q(*bad, 0) == BAD, bad
        refused("no such gather", fb.fp8_moe_gather_workspace_size, *bad)
    call = caller(lib.fp8_moe_gather, GATHER, (16384, 2048, 139264, 8, P[0], 2048, P[1], None, None, P[2], 2048, P[3], None, 0,
                                               None, 0, P[4], need, None))
    assert call() in NOGPU and call(ws=None) == EWS and call(wsb=need - 1) == EWS and call(ws=P[4] + 8) == EALIGN


def test_combine_errors(lib):
    names = ("T", "H", "R", "k", "z", "ld", "rows", "w", "y", "odt", "stream")
    call = caller(lib.fp8_moe_combine, names, (5, 256, 512, 2, P[0], 256, P[1], P[2], P[3], 0, None))
    check(call, null=("z", "rows", "y"), fine=({"w": None}, {"odt": 1}, {"odt": 2}, {"ld": 264}),
          arg=({"odt": 3}, {"odt": -1}, {"k": 17}, {"ld": 248}, {"ld": 1 << 40}, {"T": 1 << 24}, {"R": 1 << 31}),
          dim=({"T": 0}, {"k": 0}, {"H": 130}, {"R": 500}),
          align=({"z": P[0] + 8}, {"ld": 260}, {"y": P[3] + 8}, {"rows": P[1] + 2}, {"w": P[2] + 2}))
    names = ("T", "H", "R", "k", "dy", "ldd", "z", "ldz", "rows", "src", "w", "used", "q", "ldq", "s", "qT", "ldT", "sT", "dw",
             "mode", "stream")
    call = caller(lib.fp8_moe_combine_backward, names, (5, 256, 512, 2, P[0], 256, P[1], 256, P[2], P[3], P[4], None, P[5], 256,
                                                        P[6], P[7], 512, P[8], P[9], 0, None))
    check(call, null=("dy", "z", "rows", "src", "w", "q", "s", "qT", "sT", "dw"), fine=({"mode": 1, "used": P[10]},),
          arg=({"mode": 9}, {"ldd": 248}, {"ldz": 248}, {"ldq": 240}, {"ldT": 496}, {"k": 17}, {"T": 1 << 24}),
          dim=({"T": 0}, {"H": 64, "ldd": 64}, {"R": 384 + 1}),
          align=({"dy": P[0] + 8}, {"z": P[1] + 8}, {"ldz": 260}, {"rows": P[2] + 2}, {"dw": P[9] + 2}, {"w": P[4] + 2}))


@pytest.mark.parametrize("name", ["fprop", "dgrad", "wgrad"])
def test_gemm_errors(lib, name):
    names = ("R", "N", "K", "E", "a", "sa", "b", "sb", "off", "out", "odt", "mode", "stream")
    call = caller(getattr(lib, "fp8_moe_gemm_" + name), names, (512, 256, 384, 7, P[0], P[1], P[2], P[3], P[4], P[5], 0, 0, None))
    check(call, null=("a", "sa", "b", "sb", "off", "out"), fine=({"odt": 1}, {"odt": 2}, {"mode": 1}, {"E": 1024}, {"R": 128}),
          arg=({"odt": 3}, {"mode": 2}, {"E": 1025}, {"R": 1 << 29}, {"N": 1 << 25}, {"K": 1 << 25},
               {"N": 1 << 24, "K": 1 << 16}, {"R": 1 << 28, "N": 1 << 13}),
          dim=({"R": 0}, {"R": 100}, {"N": 200}, {"K": 0}, {"E": 0}, {"E": -1}),
          align=({"a": P[0] + 8}, {"b": P[2] + 8}, {"out": P[5] + 8}, {"sa": P[1] + 2}, {"sb": P[3] + 2}, {"off": P[4] + 2}))


def test_kept_errors(lib):
    names = ("M", "I", "gu", "ld", "used", "q", "ldq", "s", "qc", "ldc", "sc", "mode", "stream")
    call = caller(lib.fp8_gated_forward, names, (5, 256, P[0], 512, None, P[1], 256, P[2], P[3], 512, P[4], 0, None))
    check(call, null=("gu", "q", "s", "qc", "sc"), fine=({"qc": None, "sc": None, "ldc": 0}, {"used": P[5], "mode": 1}),
          arg=({"mode": 2}, {"ld": 504}, {"ldq": 240}, {"ldc": 496}, {"M": 1 << 31}, {"M": 1 << 29}, {"M": BIG}),
          dim=({"M": 0}, {"I": 100}),
          align=({"gu": P[0] + 8}, {"ld": 516}, {"q": P[1] + 8}, {"qc": P[3] + 8}, {"ldc": 520}, {"s": P[2] + 2},
                 {"sc": P[4] + 2}, {"used": P[5] + 2}))
    names = ("M", "I", "dh", "ld", "qc", "ldc", "sc", "used", "q", "ldq", "s", "qT", "ldT", "sT", "qh", "ldh", "sh", "mode",
             "stream")
    call = caller(lib.fp8_gated_backward, names, (384, 256, P[0], 256, P[1], 512, P[2], None, P[3], 512, P[4], P[5], 384, P[6],
                                                  P[7], 384, P[8], 0, None))
    check(call, null=("dh", "qc", "sc", "q", "s", "qT", "sT", "qh", "sh"), fine=({"used": P[9], "mode": 1},),
          arg=({"mode": 2}, {"ld": 248}, {"ldc": 496}, {"ldq": 496}, {"ldT": 368}, {"ldh": 368}, {"M": 1 << 31}),
          dim=({"M": 0}, {"M": 100}, {"I": 100}),
          align=({"dh": P[0] + 8}, {"ld": 260}, {"qc": P[1] + 8}, {"qT": P[5] + 8}, {"qh": P[7] + 8}, {"ldh": 392},
                 {"sh": P[8] + 2}, {"used": P[9] + 2}))
    names = ("q", "rows", "cols", "ld", "s", "used", "qT", "ldT", "sT", "mode", "stream")
    call = caller(lib.fp8_requantize_colgroup, names, (P[0], 256, 384, 384, P[1], None, P[2], 256, P[3], 0, None))
    check(call, null=("q", "s", "qT", "sT"), fine=({"used": P[4], "mode": 1},),
          arg=({"mode": 5}, {"ld": 368}, {"ldT": 240}, {"rows": 1 << 31, "ldT": 1 << 31}, {"ld": 1 << 40},
               {"rows": 1 << 29, "ldT": 1 << 29}),
          dim=({"rows": 100}, {"cols": 0}), align=({"q": P[0] + 8}, {"ld": 392}, {"qT": P[2] + 8}, {"s": P[1] + 2}))


def test_header_is_c(tmp_path):
    if shutil.which("gcc") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no gcc or no HIP headers")
    src, exe = tmp_path / "c.c", str(tmp_path / "c")
    src.write_text('#include "fp8train.h"\n#include <stdio.h>\nint main(void) {\n'
                   "  if (fp8_moe_sorted_rows(7, 8, 2) != 1536) return 1;\n"
                   "  if (fp8_moe_sort_workspace_size(0, 8, 2) != (size_t)-1) return 2;\n"
                   "  if (fp8_moe_sort(1, 1, 1, 0, 0, 0, 0, 0, 0, 0) != FP8BLK_ERR_NULL) return 3;\n"
                   "  if (fp8_moe_gather(1, 128, 128, 1, 0, 128, 0, 0, 0, 0, 128, 0, 0, 0, 0, 7, 0, 0, 0) != FP8BLK_ERR_ARG) return 4;\n"
                   "  if (fp8_moe_combine(1, 128, 128, 1, 0, 128, 0, 0, 0, 0, 0) != FP8BLK_ERR_NULL) return 5;\n"
                   "  if (fp8_moe_combine_backward(1, 128, 128, 1, 0, 128, 0, 128, 0, 0, 0, 0, 0, 128, 0, 0, 128, 0, 0, 0, 0) "
                   "!= FP8BLK_ERR_NULL) return 6;\n"
                   "  if (fp8_moe_gemm_fprop(128, 128, 128, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0) != FP8BLK_ERR_NULL) return 7;\n"
                   "  if (fp8_moe_gemm_dgrad(128, 128, 128, 1, 0, 0, 0, 0, 0, 0, 9, 0, 0) != FP8BLK_ERR_ARG) return 8;\n"
                   "  if (fp8_moe_gemm_wgrad(128, 128, 128, 1, 0, 0, 0, 0, 0, 0, 0, 9, 0) != FP8BLK_ERR_ARG) return 9;\n"
                   "  if (fp8_gated_forward(1, 128, 0, 256, 0, 0, 128, 0, 0, 0, 0, 0, 0) != FP8BLK_ERR_NULL) return 10;\n"
                   "  if (fp8_gated_backward(128, 128, 0, 128, 0, 256, 0, 0, 0, 256, 0, 0, 128, 0, 0, 128, 0, 0, 0) != "
                   "FP8BLK_ERR_NULL) return 11;\n"
                   "  if (fp8_requantize_colgroup(0, 128, 128, 128, 0, 0, 0, 128, 0, 0, 0) != FP8BLK_ERR_NULL) return 12;\n"
                   '  puts("ok");\n  return 0;\n}\n')
    libdir = os.path.dirname(fb.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-isystem", "/opt/rocm/include", str(src), "-o", exe, "-L", libdir,
                    "-l:libfp8blk.so", f"-Wl,-rpath,{libdir}"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)


# ------------------------------------------------------------- the binding --

class NoLibrary:
    """Stands in for the library: size queries answer, a launch fails the test."""

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 64
        if name == "fp8_moe_sorted_rows":
            return lambda *a: 512
        return lambda *a: pytest.fail("the C library was reached with bad operands")


@pytest.fixture
def host_stand_ins(monkeypatch):
    from blockwise_fp8_linear_amd import moe
    monkeypatch.setattr(train, "_functions", NoLibrary)
    for m in (moe, train):
        monkeypatch.setattr(m, "_index", lambda x, name: -1 if isinstance(x, torch.Tensor) else pytest.fail(name))
    monkeypatch.setattr(train, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(train, "_sort_sizes", lambda T, E, k: (512, 64))
    monkeypatch.setattr(train, "_gather_need", lambda *a: 64)


def test_binding_sorted(host_stand_ins):
    T, H, R, k, E = 5, 256, 512, 2, 8
    ids, rows, source, w = z((T, k), i32), z((T, k), i32), z((R,), i32), z((T, k), f32)
    x, zz = z((T, H), bf16), z((R, H), bf16)
    refused("ids: expected torch.int32", fb.fp8_moe_sort, z((T, k), torch.int64), E)
    refused("ids: expected a 2-dim", fb.fp8_moe_sort, z((T,), i32), E)
    refused("ids: must be contiguous", fb.fp8_moe_sort, z((k, T), i32).t(), E)
    refused("rows: expected shape", fb.fp8_moe_sort, ids, E, rows=z((T, 3), i32))
    refused("source: expected shape", fb.fp8_moe_sort, ids, E, source=z((R - 1,), i32))
    refused("offsets: expected shape", fb.fp8_moe_sort, ids, E, offsets=z((E,), i32))
    refused("workspace", fb.fp8_moe_sort, ids, E, workspace=3)
    refused("x: expected", fb.fp8_moe_gather, z((T, H), f32), source, k)
    refused("source: expected a 1-dim", fb.fp8_moe_gather, x, rows, k)
    refused("source: expected torch.int32", fb.fp8_moe_gather, x, source.long(), k)
    refused("weights: expected shape", fb.fp8_moe_gather, x, source, k, weights=z((T, 3), f32))
    refused("used: expected shape", fb.fp8_moe_gather, x, source, k, used=z((2,), i32))
    refused("used: expected torch.int32", fb.fp8_moe_gather, x, source, k, used=z((1,), torch.int64))
    refused("q: expected shape", fb.fp8_moe_gather, x, source, k, q=z((R, H + 128), u8))
    refused("scales of q: expected shape", fb.fp8_moe_gather, x, source, k, s=z((R, 1), f32))
    refused("qT: the last", fb.fp8_moe_gather, x, source, k, transpose=True, qT=z((R, H), u8).t())
    refused("scales of qT: must be contiguous", fb.fp8_moe_gather, x, source, k, transpose=True, sT=z((R // 128, H), f32).t())
    refused("topk", fb.fp8_moe_gather, x, source, 2 ** 32 + 2)
    refused("workspace", fb.fp8_moe_gather, x, source, k, workspace=3)
    refused("z: expected", fb.fp8_moe_combine, z((R, H), f32), rows)
    refused("rows: expected torch.int32", fb.fp8_moe_combine, zz, rows.long())
    refused("weights: expected shape", fb.fp8_moe_combine, zz, rows, z((T + 1, k), f32))
    refused("out: expected shape", fb.fp8_moe_combine, zz, rows, out=z((T, H + 1), bf16))
    refused("accumulate", fb.fp8_moe_combine, zz, rows, accumulate=True)
    refused("out_dtype", fb.fp8_moe_combine, zz, rows, out_dtype=torch.float16)
    back = fb.fp8_moe_combine_backward
    refused("z: expected shape", back, x, z((R, H + 128), bf16), rows, source, w)
    refused("rows: expected shape", back, x, zz, z((T + 1, k), i32), source, w)
    refused("source: expected shape", back, x, zz, rows, z((R - 128,), i32), w)
    refused("weights: expected torch.float32", back, x, zz, rows, source, w.bfloat16())
    refused("dweights: expected shape", back, x, zz, rows, source, w, dweights=z((T, 3), f32))


def test_binding_gemm(host_stand_ins):
    R, N, K, E = 512, 256, 384, 3
    off = z((E + 1,), i32)
    x, sx, dy, sdy = z((R, K), u8), z((R, 3), f32), z((R, N), u8), z((R, 2), f32)
    qw, sw = z((E, N, K), u8), z((E, 2, 3), f32)
    for f, a, sa in ((fb.fp8_moe_gemm_fprop, x, sx), (fb.fp8_moe_gemm_dgrad, dy, sdy)):
        refused("expected shape", f, a[:, 128:], sa, qw, sw, off)
        refused("must be contiguous", f, a.t().contiguous().t(), sa, qw, sw, off)
        refused("expected shape", f, a, sa[1:], qw, sw, off)
        refused("qw: expected a 3-dim", f, a, sa, qw[0], sw, off)
        refused("sw: expected shape", f, a, sa, qw, sw[:2], off)
        refused("offsets: expected shape", f, a, sa, qw, sw, off[1:])
        refused("offsets: expected torch.int32", f, a, sa, qw, sw, off.long())
        refused("out: expected shape", f, a, sa, qw, sw, off, out=z((R, 128), bf16))
        refused("accumulate", f, a, sa, qw, sw, off, accumulate=True)
    g = fb.fp8_moe_gemm_wgrad
    dyT, sdyT, xT, sxT = z((N, R), u8), z((N, 4), f32), z((K, R), u8), z((K, 4), f32)
    refused("qxT: expected shape", g, dyT, sdyT, xT[:, 128:], sxT, off)
    refused("sdyT: expected shape", g, dyT, sdyT[:, 1:], xT, sxT, off)
    refused("sxT: expected torch.float32", g, dyT, sdyT, xT, sxT.double(), off)
    refused("2-dim", g, dyT[None], sdyT, xT, sxT, off)
    refused("offsets: expected a 1-dim", g, dyT, sdyT, xT, sxT, off[None])
    refused("offsets: expected a 1-dim", g, dyT, sdyT, xT, sxT, off[:1])
    refused("out: expected shape", g, dyT, sdyT, xT, sxT, off, out=z((E, K, N), bf16))


def test_binding_kept(host_stand_ins):
    M, I = 256, 384
    gu, dh, qc, sc = z((M, 2 * I), bf16), z((M, I), bf16), z((M, 2 * I), u8), z((M, 6), f32)
    refused("gu: expected", fb.fp8_gated_forward, z((M, 2 * I), f32))
    refused("gu: expected", fb.fp8_gated_forward, z((M, 5), bf16))
    refused("qc: expected shape", fb.fp8_gated_forward, gu, qc=z((M, I), u8))
    refused("scales of q: expected shape", fb.fp8_gated_forward, gu, s=z((M, 6), f32))
    refused("qc: expected shape", fb.fp8_gated_backward, dh, z((M, I), u8), z((M, 3), f32))
    refused("scales of qc: expected shape", fb.fp8_gated_backward, dh, qc, sc[:, :3])
    refused("qhT: expected shape", fb.fp8_gated_backward, dh, qc, sc, qhT=z((2 * I, M), u8))
    refused("used: expected", fb.fp8_gated_backward, dh, qc, sc, used=7)
    refused("q: expected torch.uint8", fb.fp8_requantize_colgroup, qc.to(torch.int8), sc)
    refused("scales of q: expected shape", fb.fp8_requantize_colgroup, qc, sc[:128])
    refused("qT: expected shape", fb.fp8_requantize_colgroup, qc, sc, qT=z((M, 2 * I), u8))


def test_binding_refuses_host_tensors():
    for fn, args in ((fb.fp8_moe_sort, (z((1, 2), i32), 4)), (fb.fp8_moe_gather, (z((1, 128), bf16), z((128,), i32), 1)),
                     (fb.fp8_moe_combine, (z((128, 128), bf16), z((1, 1), i32))),
                     (fb.fp8_moe_gemm_fprop, (z((128, 128), u8), None, None, None, None)),
                     (fb.fp8_gated_forward, (z((1, 256), bf16),)), (fb.fp8_requantize_colgroup, (z((128, 128), u8), None))):
        refused("device tensor", fn, *args)


def test_host_checks_under_sanitizers(tmp_path):
    """api_train.cpp under gcc's address and undefined-behaviour sanitizers, its launchers replaced by stubs that hold what
    each would read and write against what the sizes say."""
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no g++ or no HIP headers")
    csrc, exe = os.path.join(ROOT, "blockwise_fp8_linear_amd", "csrc"), str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                    "-isystem", "/opt/rocm/include", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "api_train_host_check.cpp"),
                    os.path.join(csrc, "api_train.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-4000:] + r.stderr[-4000:]


def test_grouped_wgrad_uses_no_scratch(tmp_path):
    """grouped_wgrad.hip counts on its registers: a spill would go through memory beside its direct loads."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc) and shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    out = str(tmp_path / "grouped_wgrad.s")
    subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Wno-inline-asm", "-Wno-unused-function",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"),
                    "--cuda-device-only", "-S", "-o", out,
                    os.path.join(ROOT, "blockwise_fp8_linear_amd", "csrc", "grouped_wgrad.hip")],
                   check=True, capture_output=True, text=True)
    text = open(out).read()
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)
    assert sizes and all(int(s) == 0 for s in sizes) and "scratch_" not in text
