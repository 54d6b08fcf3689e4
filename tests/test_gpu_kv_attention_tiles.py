"""Attention over the E4M3 cache on the tcgen05 kernel. Which kernel a call
takes depends on all its sizes, so every test here asks for the plan and fails
if its call does not reach that kernel."""
import math

import pytest
import torch

import attention_reference as ref
from test_gpu_kv_attention import filled
from test_gpu_kv_cache import ints, offsets_of

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("dit_rowwise_amax_b200")

OK, INDEX = 0, 6


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_len", [0, 1, 20])
def test_rows_that_see_nothing_without_key_ranges(dim, kv_len):
    """More new tokens than cached ones under a causal mask, up to none cached
    at all: slots without a key tile still write zeros (and -inf), not what
    their Q buffer holds. One range of keys, so nothing is joined afterwards.
    Many times over, since a slot's warps arrive in any order."""
    g = torch.Generator("cuda").manual_seed(dim + kv_len)
    requests, heads, new, t = 16, 8, 512, 128
    cache = filled(3, t, heads, dim, g)
    offs = offsets_of([new] * requests)
    table = [[1] + [1 << 30] * 7] * requests
    ints_ = (ints(table), ints([kv_len] * requests), ints(offs))
    q = torch.randn((offs[-1], heads, dim), generator=g, device="cuda").bfloat16()
    rows, cut = fp8.kv_cache_attention_plan(q, cache, *ints_, max_q=new)
    assert (rows, cut) == (256, 1)
    want, want_lse, bound, _ = ref.attention(q[:new], cache, [[1]], [kv_len], [0, new], dim ** -0.5, 1)
    for turn in range(25):
        out = torch.full_like(q, 7.0)
        _, lse = fp8.kv_cache_attention(q, cache, *ints_, max_q=new, causal=1, out=out, return_lse=True)
        unseen = new - kv_len
        out, lse = out.view(requests, new, heads, dim), lse.view(requests, new, heads)
        assert bool((out[:, :unseen] == 0).all()) and bool((lse[:, :unseen] == -math.inf).all()), turn
        assert bool(((out[0].double() - want).abs() <= bound).all()) and torch.equal(lse[0].isinf(), want_lse.isinf())
    assert fp8.device_error() == OK
