"""Refusals of the attention operators, through the C-ABI and the Python
binding. Every argument is checked before a device is touched, so these run
without a GPU; the pointers are host memory that nothing reads."""
import ctypes

import pytest
import torch

import dit_rowwise_amax_b200 as fp8

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from dit_rowwise_amax_b200 import build
    build.build()
    return fp8.load_library()


BUF = (ctypes.c_uint8 * 4096)()
PTR = (ctypes.addressof(BUF) + 63) // 64 * 64


def heads(n=4, dim=64, **kw):
    a = dict(ptr=PTR, token_stride=n * dim, head_stride=dim, heads=n, reserved=0)
    a.update(kw)
    return fp8._Heads(*a.values())


def rotary(lib, q=None, k=None, qo=None, ko=None, M=2, dim=64, pos=PTR, kind=0, freqs=None, dims=(32, 32), interleaved=1):
    f = (ctypes.c_double * 128)(*([1.0] * 128)) if freqs is None else freqs
    none = fp8._Heads(None, 0, 0, 0, 0)
    return lib.fp8_rotary_axes(q or heads(dim=dim), k or none, qo or heads(dim=dim), ko or none, M, dim, pos, kind, f,
                               (ctypes.c_int32 * max(len(dims), 1))(*dims), len(dims), interleaved, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(M=-1), INVALID), (dict(dim=60, dims=(32,)), UNSUPPORTED), (dict(dim=264, dims=(32,)), UNSUPPORTED),
    (dict(dim=0), UNSUPPORTED), (dict(dims=()), UNSUPPORTED), (dict(dims=(2,) * 5), UNSUPPORTED), (dict(dims=(3,)), UNSUPPORTED),
    (dict(dims=(0, 8)), UNSUPPORTED), (dict(dims=(-2,)), UNSUPPORTED), (dict(dims=(32, 34)), UNSUPPORTED),
    (dict(dims=(2 ** 31 - 2, 2 ** 31 - 2)), UNSUPPORTED), (dict(dims=(4,), interleaved=0), UNSUPPORTED), (dict(kind=2), INVALID),
    (dict(pos=None), INVALID), (dict(pos=PTR + 2), INVALID), (dict(q=heads(ptr=None)), INVALID), (dict(q=heads(ptr=PTR + 8)), INVALID),
    (dict(q=heads(token_stride=60)), INVALID), (dict(q=heads(token_stride=0)), INVALID), (dict(q=heads(head_stride=32)), INVALID),
    (dict(q=heads(head_stride=68)), INVALID), (dict(q=heads(reserved=1)), INVALID), (dict(q=heads(5)), INVALID),
    (dict(q=heads(-1), qo=heads(-1)), INVALID), (dict(k=heads(2)), INVALID), (dict(k=heads(2, ptr=None), ko=heads(2)), INVALID),
    (dict(freqs=(ctypes.c_double * 128)(*([float("inf")] * 128))), INVALID), (dict(M=2 ** 31), UNSUPPORTED),
])
def test_rotary_refusals(lib, kw, want):
    assert rotary(lib, **kw) == want
    assert (lib.fp8dit_last_error_string() == b"") == (want == OK)


def cache(**kw):
    a = dict(k=PTR, v=PTR, ks=PTR, vs=PTR, n_blocks=8, kv_heads=2, block_tokens=16, head_dim=64)
    a.update(kw)
    return fp8._KvCache(*a.values())


def batch(**kw):
    a = dict(table=PTR, lens=PTR, offsets=PTR, total=4, n=2, width=3, max_new=2, max_kv=40)
    a.update(kw)
    return fp8._KvBatch(*a.values())


CACHE = [(dict(k=None), INVALID), (dict(v=PTR + 8), INVALID), (dict(ks=None), INVALID), (dict(vs=PTR + 2), INVALID),
         (dict(n_blocks=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=65536), UNSUPPORTED), (dict(block_tokens=8), UNSUPPORTED),
         (dict(block_tokens=256), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED)]
BATCH = [(dict(n=-1), INVALID), (dict(total=-1), INVALID), (dict(max_new=-1), INVALID), (dict(max_kv=-1), INVALID),
         (dict(width=-1), INVALID), (dict(max_kv=49), INVALID), (dict(n=65536), UNSUPPORTED), (dict(total=2 ** 31), UNSUPPORTED),
         (dict(lens=None), INVALID), (dict(offsets=None), INVALID), (dict(table=None), INVALID), (dict(offsets=PTR + 1), INVALID),
         (dict(n=0), OK), (dict(total=0), OK), (dict(max_new=0), OK)]


@pytest.mark.parametrize("c,b,want", [(c, {}, w) for c, w in CACHE] + [({}, b, w) for b, w in BATCH])
def test_cache_and_batch_refusals(lib, c, b, want):
    x = cache(**c)
    assert lib.fp8_kv_cache_append(x, heads(2), heads(2), batch(**b), None) == want
    assert lib.fp8_kv_cache_attention(x, heads(4), batch(**b), heads(4), None, 0.125, 0, None, 0, None) == want
    assert lib.fp8_kv_cache_attention_workspace_size(x, batch(**b), 4) == 0


def test_append_refusals(lib):
    for k, v, want in ((heads(3), heads(2), INVALID), (heads(2), heads(2, ptr=None), INVALID), (heads(2, token_stride=100), heads(2), INVALID)):
        assert lib.fp8_kv_cache_append(cache(), k, v, batch(), None) == want
    assert lib.fp8_kv_cache_append(None, heads(2), heads(2), batch(), None) == INVALID
    assert lib.fp8_kv_cache_append(cache(), heads(2), heads(2), None, None) == INVALID
    big = batch(n=65535, max_new=2 ** 30, total=2 ** 30)
    assert lib.fp8_kv_cache_append(cache(), heads(2), heads(2), big, None) == UNSUPPORTED


def attend(lib, q=None, out=None, lse=None, scale=0.125, causal=0, b=None):
    return lib.fp8_kv_cache_attention(cache(), q or heads(4), b or batch(), out or heads(4), lse, scale, causal, None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=heads(3), out=heads(3)), INVALID), (dict(q=heads(0), out=heads(0)), INVALID), (dict(out=heads(2)), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(causal=-1), INVALID), (dict(lse=PTR + 2), INVALID), (dict(out=heads(4, ptr=PTR + 4)), INVALID),
    (dict(q=heads(4, head_stride=4)), INVALID), (dict(q=heads(65538), out=heads(65538)), UNSUPPORTED),
    (dict(b=batch(max_new=2 ** 30)), UNSUPPORTED),
])
def test_attention_refusals(lib, kw, want):
    assert attend(lib, **kw) == want


def test_python_refuses_host_and_wrong_tensors():
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp8.rotary_axes(q, None, torch.zeros((4, 1), dtype=torch.int32), fp8.rotary_frequencies((64,)), (64,))
    with pytest.raises(ValueError):
        fp8.rotary_axes(q.float(), None, torch.zeros((4, 1), dtype=torch.int32), fp8.rotary_frequencies((64,)), (64,))
    c = fp8.KVCache.empty(2, 16, 2, 64, device="cpu")
    ints = [torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)]
    with pytest.raises(ValueError):
        fp8.kv_cache_append(c, q, q, *ints, max_new=1)
    with pytest.raises(ValueError):
        fp8.kv_cache_attention(q, c, *ints, max_q=1)


def test_python_refuses_bounds_beyond_32_bits():
    cpu = torch.device("cpu")
    ints = [torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)]
    for new, kv in ((1 << 32, 16), (-1, 16), (1, 1 << 32), (1, -1)):
        with pytest.raises(ValueError):
            fp8._kv_batch(*ints, 1, new, kv, 16, cpu)
    assert fp8._kv_batch(*ints, 1, 1, None, 16, cpu).max_kv == 32
    wide = torch.zeros((1, 1), dtype=torch.int32).expand(1, 1 << 26)  # 2^33 tokens: the default bound is cut to 2^30
    with pytest.raises(ValueError):
        fp8._kv_batch(wide, *ints[1:], 1, 1, None, 128, cpu)  # not contiguous
    with pytest.raises(ValueError):
        fp8._kv_batch(ints[0].long(), *ints[1:], 1, 1, None, 16, cpu)
    with pytest.raises(ValueError):
        fp8._kv_batch(ints[0], ints[1], ints[1], 1, 1, None, 16, cpu)


def test_rotary_frequencies():
    f = fp8.rotary_frequencies((4, 8), 100.0)
    want = [1.0, 100.0 ** -0.5, 1.0, 100.0 ** -0.25, 100.0 ** -0.5, 100.0 ** -0.75]
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-15)
