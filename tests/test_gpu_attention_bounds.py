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


@pytest.mark.parametrize("new,kernel", [(1, 8), (100, 256)])
@pytest.mark.parametrize("dim", [64, 128])
def test_values_near_the_largest_through_joined_ranges(new, kernel, dim):
    """Four ranges or more of equal weight, every value 1.9 2^126: their sum is
    beyond fp32, their mean is not."""
    t, n = 128, 40960
    cache = filled(2, t, 1, dim, torch.Generator("cuda").manual_seed(2))
    cache.v.fill_(0x77)  # 240
    cache.v_scale.fill_(2.0 ** 119)
    q = torch.zeros((new, 1, dim), dtype=torch.bfloat16, device="cuda")
    args = (q, cache, ints([[0, 1] * (n // t // 2)]), ints([n]), ints([0, new]))
    rows, ranges = fp8.kv_cache_attention_plan(*args, max_q=new)
    assert rows == kernel and ranges >= 4
    out = fp8.kv_cache_attention(*args, max_q=new)
    # sums of up to n equal terms are exact; the division, the join's weights and products: 2^-20
    assert bool(((out.double() / (240 * 2.0 ** 119) - 1).abs() <= 2.0 ** -8 + 2.0 ** -20).all())
    assert fp8.device_error() == OK
