"""The query of an attention call's plan: refusals and calls without rows (no
GPU), and its agreement with the workspace query."""
import ctypes

import pytest
import torch

import dit_rowwise_amax_b200 as fp8
from test_attention_args import BATCH, CACHE, INVALID, OK, UNSUPPORTED, batch, cache


@pytest.fixture(scope="module")
def lib():
    from dit_rowwise_amax_b200 import build
    build.build()
    return fp8.load_library()


def plan(lib, c, b, q_heads=4):
    rows, ranges = ctypes.c_int32(-1), ctypes.c_int32(-1)
    return lib.fp8_kv_cache_attention_plan(c, b, q_heads, ctypes.byref(rows), ctypes.byref(ranges)), rows.value, ranges.value


@pytest.mark.parametrize("c,b,want", [(c, {}, w) for c, w in CACHE]
                         + [({}, b, w) for b, w in BATCH if "lens" not in b and "offsets" not in b and "table" not in b])
def test_plan_refusals(lib, c, b, want):
    status, rows, ranges = plan(lib, cache(**c), batch(**b))
    assert status == want
    assert (rows, ranges) == ((0, 0) if want == OK else (-1, -1))


def test_plan_refuses_heads(lib):
    for heads in (0, -2, 3):
        assert plan(lib, cache(), batch(), heads)[0] == INVALID
    assert lib.fp8_kv_cache_attention_plan(None, batch(), 4, None, None) == INVALID
    assert lib.fp8_kv_cache_attention_plan(cache(), None, 4, None, None) == INVALID
    assert lib.fp8_kv_cache_attention_plan(cache(), batch(n=0), 4, None, None) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("requests,new,heads,kv,cached", [(1, 1, 16, 16, 26), (32, 1, 32, 8, 16001), (3, 4, 8, 2, 900), (1, 5, 8, 2, 40),
                                                          (5, 700, 24, 8, 6001), (1, 1560, 16, 16, 32760), (1, 26, 16, 16, 32760)])
def test_plan_agrees_with_the_workspace(requests, new, heads, kv, cached):
    c = fp8.KVCache.empty(4, 128, kv, 64)
    table = torch.zeros((requests, -(-cached // 128)), dtype=torch.int32, device="cuda")
    lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(requests + 1, dtype=torch.int32, device="cuda")
    q = torch.empty((requests * new, heads, 64), dtype=torch.bfloat16, device="cuda")
    rows, ranges = fp8.kv_cache_attention_plan(q, c, table, lens, offsets, max_q=new, max_kv=cached)
    per_request = new * heads // kv
    if per_request <= 16:
        assert rows == (8 if per_request <= 8 else 16)
    else:
        assert rows in (16, 256)
    desc = fp8._kv_batch(table, lens, offsets, requests * new, new, cached, 128, q.device)
    need = fp8.load_library().fp8_kv_cache_attention_workspace_size(fp8._kv_cache(c)[0], desc, heads)
    assert 1 <= ranges <= 64 and (need > 0) == (ranges > 1)


@pytest.mark.parametrize("q_heads,max_new", [(1 << 16, 2), (1 << 20, 1 << 20), (1 << 30, 1 << 30), (4, 1 << 29)])
def test_sizes_that_the_call_refuses_have_no_plan_and_no_workspace(lib, q_heads, max_new):
    b = batch(max_new=max_new, total=1 << 30)
    assert plan(lib, cache(kv_heads=1), b, q_heads)[0] == UNSUPPORTED
    assert lib.fp8_kv_cache_attention_workspace_size(cache(kv_heads=1), b, q_heads) == 0
    assert lib.fp8dit_last_error_string() != b""


def test_a_call_of_nothing_may_have_any_bound(lib):
    empty = batch(max_new=1 << 30, total=0)
    assert plan(lib, cache(kv_heads=1), empty, 4) == (OK, 0, 0)
    c, q = cache(), fp8._Heads(None, 256, 64, 4, 0)
    assert lib.fp8_kv_cache_attention(c, q, empty, q, None, 0.125, 0, None, 0, None) == OK
