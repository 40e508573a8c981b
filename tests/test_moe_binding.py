"""The binding of include/fp8moe.h on calls that the library refuses, without
a GPU: the refusal is the library's, and nothing is allocated for the call."""
import pytest
import torch

import blockwise_fp8_linear_amd as fb
from blockwise_fp8_linear_amd import moe


@pytest.fixture
def no_device(monkeypatch):
    monkeypatch.setattr(moe, "_index", lambda x, name: -1)
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(moe, "_new", lambda *a: pytest.fail("allocated for a refused call"))


@pytest.mark.parametrize("topk,status", [(17, -4), (10 ** 6, -4), (9, -4), (2 ** 31 - 1, -4), (0, -2), (-3, -2),
                                         (-2 ** 31, -2)])
def test_route_of_a_refused_topk_allocates_nothing(no_device, topk, status):
    E = 64 if topk == 17 else 8
    with pytest.raises(RuntimeError) as e:
        fb.fp8_moe_route(torch.zeros((3, E)), topk)
    assert str(e.value) == fb.fp8_status_string(status)


P = [0x100000 * i for i in range(1, 10)]    # addresses that are never read
EARG, NOGPU = -4, (-6, -7)                  # the latter where only the device is missing


@pytest.fixture
def lib():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: valid arguments would launch on these addresses")
    return moe._functions()


def _linear(lib, M, N, K, ld):
    return lib.fp8_linear(M, N, K, P[0], ld, P[1], P[2], P[3], 0, 0, P[4], 2 ** 62, None)


@pytest.mark.parametrize("at,past", [
    ((3, 128, 128, 2 ** 26), (3, 128, 128, 2 ** 26 + 8)),                    # row stride
    ((2 ** 27 - 1, 128, 128, 128), (2 ** 27, 128, 128, 128)),                # M
    ((1, 2 ** 27 - 128, 128, 128), (1, 2 ** 27, 128, 128)),                  # N
    ((1, 128, 2 ** 25 - 128, 2 ** 25), (1, 128, 2 ** 25, 2 ** 25)),          # K
    ((2 ** 20, 2 ** 20, 128, 128), (2 ** 20, 2 ** 20 + 128, 128, 128)),      # M N
    ((1, 2 ** 20, 2 ** 20, 2 ** 20), (1, 2 ** 20 + 128, 2 ** 20, 2 ** 20)),  # N K
    ((2 ** 15, 128, 128, 2 ** 25), (2 ** 15 + 1, 128, 128, 2 ** 25)),        # M ld
])
def test_linear_takes_what_the_header_says(lib, at, past):
    assert _linear(lib, *at) in NOGPU
    assert _linear(lib, *past) == EARG


def test_route_and_mixture_take_what_the_header_says(lib):
    def route(T, ld):
        return lib.fp8_moe_route(T, 4, 2, P[0], 0, ld, 1, P[1], P[2], None)

    def experts(T, H, I, k, ld):
        return lib.fp8_moe_experts(T, H, I, 16, k, P[0], ld, P[1], P[2], P[3], P[4], P[5], P[6], P[7], 0, 0, P[8],
                                   2 ** 62, None)
    assert route(2 ** 31 - 1, 4) in NOGPU and route(2 ** 31, 4) == EARG
    assert route(2 ** 20, 2 ** 20) in NOGPU and route(2 ** 20, 2 ** 20 + 1) == EARG
    for at, past in (((2, 128, 128, 1, 2 ** 26), (2, 128, 128, 1, 2 ** 26 + 8)),                    # row stride
                     ((2, 2 ** 20, 512, 1, 2 ** 20), (2, 2 ** 20 + 128, 128, 1, 2 ** 21)),          # H
                     ((2, 512, 2 ** 20, 1, 512), (2, 128, 2 ** 20 + 128, 1, 512)),                  # I
                     ((2, 2 ** 15, 2 ** 14, 1, 2 ** 15), (2, 2 ** 15, 2 ** 14 + 128, 1, 2 ** 15)),  # H I
                     ((512, 128, 2 ** 18 - 128, 16, 128), (512, 128, 2 ** 18, 16, 128))):           # T k I
        assert experts(*at) in NOGPU and experts(*past) == EARG, (at, past)
