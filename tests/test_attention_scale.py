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


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["few rows", "copies", "loose"])
@pytest.mark.parametrize("exponent", [20, 23, 26, 29, 33, 60])
@pytest.mark.parametrize("spread", [0, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_so_large_that_one_key_takes_all(how, exponent, spread, sign):
    """Scores near +-2^exponent (log2 units), at least 2^(exponent - 18) apart or
    equal: a row's output is the mean value of its largest keys. With
    spread, V's block scales differ by as much too."""
    from test_gpu_kv_attention import filled
    from test_gpu_kv_attention_tiles import attend as attend_tiles
    from test_gpu_kv_attention_tiles import sizes_for_tiles
    from test_gpu_kv_cache import ints
    import attention_reference as ref
    import math
    g = torch.Generator("cuda").manual_seed(exponent)
    dim, t, n, new = 64, 32, 600, 7 if how == "few rows" else 150
    blocks = -(-n // t)
    cache = filled(blocks, t, 1, dim, g)
    cache.v_scale.copy_(torch.exp2(-torch.randint(0, spread + 1, (blocks, 1), generator=g, device="cuda").float()))
    cache.k.zero_()
    cache.k_scale.fill_(2.0 ** (exponent - 40))
    cache.k[..., 0] = 0x38 if sign > 0 else 0xB8  # +-1
    cache.k[..., 1] = torch.randint(0x38, 0x48, cache.k.shape[:3], generator=g, device="cuda").to(torch.uint8)  # 1 .. 3.75 in steps
    q = torch.zeros((new, 1, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** 40
    q[..., 1] = torch.exp2(torch.randint(25, 40, (new, 1), generator=g, device="cuda").float()).bfloat16()
    scale = 1.37 * math.log(2.0)
    pages = list(range(blocks))
    if how == "few rows":
        out = fp8.kv_cache_attention(q, cache, ints([pages]), ints([n]), ints([0, new]), max_q=new, scale=scale)
    else:
        copies, width = sizes_for_tiles(1, cache, [pages], [n], [0, new], how)
        out, _ = attend_tiles(q, cache, [pages], [n], [0, new], copies, width, 0, scale)
    values = ref.e4m3_table("cuda")
    k = (values[cache.k.long()] * cache.k_scale.double()[:, :, None, None])[:, 0].reshape(-1, dim)[:n]
    v = (values[cache.v.long()] * cache.v_scale.double()[:, :, None, None])[:, 0].reshape(-1, dim)[:n]
    s = q[:, 0].double() @ k.T
    best = (s == s.amax(1, keepdim=True)).double()
    gap = (s.amax(1, keepdim=True) - s)[best == 0].min() * 1.37
    assert gap >= 2.0 ** (exponent - 18)
    p = best / best.sum(1, keepdim=True)
    # equal weights, and what the others may weigh at a gap of 4 or more in log2 units
    rest = n * 2.0 ** -float(gap) * v.abs().max()
    bound = 1.01 * 2.0 ** -8 * (p @ v).abs() + (2.0 ** -11 + n * 2.0 ** -23) * (p @ v.abs()) + rest
    err = (out[:, 0].double() - p @ v).abs()
    assert bool((err <= bound).all()), (float((err / bound.clamp(min=1e-300)).max()), bool(err.isnan().any()))
    assert fp8.device_error() == 0
