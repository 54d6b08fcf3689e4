"""Softmax scales, queries and key scales at the ends of their ranges."""
import pytest
import torch

import dit_rowwise_amax_b200 as fp8
from test_attention_args import INVALID, attend


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_refuses_scales_that_leave_the_range_in_log2_units(scale):
    from dit_rowwise_amax_b200 import build
    build.build()
    assert attend(fp8.load_library(), scale=scale) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["few rows", "copies", "loose"])
@pytest.mark.parametrize("scale,q_exponent,k_exponent", [(2.0 ** -20, -110, 118), (2.0 ** -40, -80, 110), (2.0 ** -100, -26, 118),
                                                         (2.0 ** 100, -112, 4), (2.0 ** -120, 112, 0), (0.125, 0, -9)])
def test_small_queries_and_scales_under_large_keys(scale, q_exponent, k_exponent, how):
    """scale q k is near one throughout, its parts are not."""
    from test_gpu_kv_attention import check, filled
    from test_gpu_kv_attention_tiles import check_seen
    g = torch.Generator("cuda").manual_seed(30)
    heads, dim, t, n = 1, 64, 32, 200
    cache = filled(7, t, heads, dim, g)
    cache.k_scale.fill_(2.0 ** k_exponent)
    cache.k_scale[::2] *= 0.25
    new = 9 if how == "few rows" else 150
    q = (torch.randn((new, heads, dim), generator=g, device="cuda") * 2.0 ** q_exponent).bfloat16()
    if how == "few rows":
        check(q, cache, [list(range(7))], [n], [0, new], 0, scale=scale, max_q=new)
    else:
        check_seen(q, cache, list(range(7)), n, scale=scale, how=how)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["few rows", "copies"])
def test_large_factors_of_a_product_of_zero(how):
    """q's one large element meets zeros: every score is 0, though scale x |q| x
    K's block scale is beyond fp32."""
    from test_gpu_kv_attention import filled
    from test_gpu_kv_attention_tiles import attend as attend_tiles
    from test_gpu_kv_attention_tiles import sizes_for_tiles
    from test_gpu_kv_cache import ints
    dim, t, n = 64, 16, 100
    cache = filled(7, t, 1, dim, torch.Generator("cuda").manual_seed(31))
    cache.k[..., 3] = 0
    cache.k_scale.fill_(2.0 ** 60)
    new = 5 if how == "few rows" else 150
    q = torch.zeros((new, 1, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 3] = 2.0 ** 127
    if how == "few rows":
        out = fp8.kv_cache_attention(q, cache, ints([list(range(7))]), ints([n]), ints([0, new]), max_q=new)
    else:
        copies, width = sizes_for_tiles(1, cache, [list(range(7))], [n], [0, new], how)
        out, _ = attend_tiles(q, cache, [list(range(7))], [n], [0, new], copies, width, 0, 0.125)
    import attention_reference as ref
    v = (ref.e4m3_table("cuda")[cache.v.long()] * cache.v_scale.double()[:, :, None, None])[:, 0].reshape(-1, dim)[:n]
    # equal weights; n fp32 additions and a weight's 2^-22
    bound = 2.0 ** -8 * v.mean(0).abs() + (n * 2.0 ** -23 + 2.0 ** -21) * v.abs().mean(0)
    assert bool(((out[:, 0].double() - v.mean(0)).abs() <= bound).all())
