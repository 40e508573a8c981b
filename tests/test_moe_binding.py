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
