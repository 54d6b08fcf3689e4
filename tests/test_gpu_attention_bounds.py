"""Bounds of a call's sizes that its device numbers break, or that say there is
nothing to do."""
import pytest
import torch

import attention_reference as ref
from test_gpu_kv_attention import filled
from test_gpu_kv_cache import ints

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("dit_rowwise_amax_b200")

OK, INDEX = 0, 6


@pytest.mark.parametrize("offsets,reported", [([0, 0, 0], False), ([0, 2, 2], True), ([0, 0, 5], True)])
def test_a_bound_of_no_new_tokens_is_checked(offsets, reported):
    """max_new = max_q = 0: a request with several new tokens is left out and
    reported, one without any is not, and nothing is written."""
    cache = filled(4, 16, 1, 64, torch.Generator("cuda").manual_seed(1))
    before = [x.clone() for x in cache]
    q = torch.ones((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    args = (ints([[0, 1], [2, 3]]), ints([8, 9]), ints(offsets))
    out = torch.full_like(q, 7.0)
    fp8.kv_cache_attention(q, cache, *args, max_q=0, out=out)
    assert fp8.device_error() == (INDEX if reported else OK)
    assert bool((out == 7.0).all())
    fp8.kv_cache_append(cache, q[:, :1], q[:, :1], *args, max_new=0)
    assert fp8.device_error() == (INDEX if reported else OK)
    assert all(torch.equal(a, b) for a, b in zip(cache, before))


def test_a_bound_of_no_new_tokens_and_one_new_token():
    cache = filled(4, 16, 1, 64, torch.Generator("cuda").manual_seed(1))
    q = torch.randn((1, 2, 64), device="cuda").bfloat16()
    out = fp8.kv_cache_attention(q, cache, ints([[0, 1]]), ints([20]), ints([0, 1]), max_q=0)
    want, _, bound, _ = ref.attention(q, cache, [[0, 1]], [20], [0, 1], 0.125, 0)
    assert bool(((out.double() - want).abs() <= bound).all()) and fp8.device_error() == OK
