"""Rotary positions with several axes against the float64 rotation. An output
is rounded to bf16 once (half a step: 2^-8 of it); sine, cosine (2 ulp each),
the angle in turns as fp32 (2^-25, times 2 pi) and the two fp32 products and
their sum are off by less than 2^-20 (|x| + |y|)."""
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("dit_rowwise_amax_b200")


def check(got, x, pos, freqs, dims, interleaved):
    want = ref.rotary(x, pos, freqs, dims, interleaved)
    p = freqs.numel()
    mass = x.double().abs()
    a, b = (slice(0, 2 * p, 2), slice(1, 2 * p, 2)) if interleaved else (slice(0, p), slice(p, 2 * p))
    pair = mass[..., a] + mass[..., b]
    tol = 2.0 ** -8 * want.abs()
    tol[..., a] += 2.0 ** -20 * pair
    tol[..., b] += 2.0 ** -20 * pair
    assert bool(((got.double() - want).abs() <= tol + 1e-38).all())
    if 2 * p < x.shape[2]:
        assert torch.equal(got[..., 2 * p:], x[..., 2 * p:])


@pytest.mark.parametrize("tokens", [1, 2, 7, 133, 4099])
@pytest.mark.parametrize("heads,kv,dim,dims", [(1, 0, 8, (8,)), (16, 16, 128, (16, 56, 56)), (5, 1, 64, (16, 24, 24)),
                                               (3, 3, 96, (32, 32, 16)), (2, 1, 256, (64, 96, 96)), (3, 2, 128, (8, 8, 8, 8))])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary(tokens, heads, kv, dim, dims, interleaved):
    g = torch.Generator("cuda").manual_seed(tokens * 31 + heads)
    q = torch.randn((tokens, heads, dim), generator=g, device="cuda").bfloat16()
    k = torch.randn((tokens, kv, dim), generator=g, device="cuda").bfloat16() if kv else None
    pos = torch.randint(-50, 5000, (tokens, len(dims)), generator=g, device="cuda", dtype=torch.int32)
    freqs = fp8.rotary_frequencies(dims, 256.0)
    qo, ko = fp8.rotary_axes(q, k, pos, freqs, dims, interleaved=interleaved)
    check(qo, q, pos, freqs, dims, interleaved)
    if kv:
        check(ko, k, pos, freqs, dims, interleaved)
    else:
        assert ko is None


@pytest.mark.parametrize("pairs", [1, 3, 5])
def test_odd_numbers_of_interleaved_pairs(pairs):
    """Rotated elements that end inside a 16-byte unit."""
    q = torch.randn((9, 3, 16), device="cuda").bfloat16()
    pos = torch.arange(9, device="cuda", dtype=torch.int32)[:, None].contiguous()
    freqs = fp8.rotary_frequencies((2 * pairs,))
    qo, _ = fp8.rotary_axes(q, None, pos, freqs, (2 * pairs,))
    check(qo, q, pos, freqs, (2 * pairs,), True)


@pytest.mark.parametrize("interleaved", [True, False])
def test_far_fractional_positions_merged_views_in_place(interleaved):
    m, hq, hk, d, dims = 517, 6, 2, 64, (16, 16)
    qkv = torch.randn((m, (hq + 2 * hk) * d), device="cuda").bfloat16()
    before = qkv.clone()
    q, k = qkv[:, : hq * d].view(m, hq, d), qkv[:, hq * d: (hq + hk) * d].view(m, hk, d)
    q0, k0 = q.clone(), k.clone()
    pos = (torch.rand((m, 2), device="cuda") * 2e6 - 1e6).float()
    freqs = fp8.rotary_frequencies(dims)
    qo, ko = fp8.rotary_axes(q, k, pos, freqs, dims, interleaved=interleaved, q_out=q, k_out=k)
    assert qo is q and ko is k
    check(q, q0, pos, freqs, dims, interleaved)
    check(k, k0, pos, freqs, dims, interleaved)
    assert torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])  # v is left alone


def test_largest_positions():
    """int32 limits: the angle is reduced in double, an fp32 product would be off by turns."""
    q = torch.randn((4, 2, 8), device="cuda").bfloat16()
    pos = torch.tensor([[2 ** 31 - 1], [-2 ** 31], [2 ** 30 + 1], [0]], dtype=torch.int32, device="cuda")
    freqs = torch.tensor([1.0, 0.1, 1e-3, 1e-7], dtype=torch.float64)
    qo, _ = fp8.rotary_axes(q, None, pos, freqs, (8,))
    # the float64 reference itself is off by 2^31 * 2^-53 here, far below the tolerance
    check(qo, q, pos, freqs, (8,), True)


def test_head_stride_other_stream_and_graph():
    x = torch.randn((40, 128, 3), device="cuda").bfloat16().permute(0, 2, 1)  # heads not contiguous: refused
    pos = torch.zeros((40, 1), dtype=torch.int32, device="cuda")
    freqs = fp8.rotary_frequencies((128,))
    with pytest.raises(ValueError):
        fp8.rotary_axes(x, None, pos, freqs, (128,))
    y = torch.randn((3, 40, 128), device="cuda").bfloat16().permute(1, 0, 2)  # [tokens, heads, dim], head-major memory
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[:, None].contiguous()
    out = torch.empty((40, 3, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fp8.rotary_axes(y, None, pos, freqs, (128,), q_out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fp8.rotary_axes(y, None, pos, freqs, (128,), q_out=out)
    torch.cuda.synchronize()
    check(out, y, pos, freqs, (128,), True)
    pos += 100
    graph.replay()
    torch.cuda.synchronize()
    check(out, y, pos, freqs, (128,), True)


def test_no_tokens():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    qo, _ = fp8.rotary_axes(q, None, pos, fp8.rotary_frequencies((64,)), (64,))
    assert qo.shape == (0, 4, 64)
