"""Attention over the E4M3 cache on the tcgen05 kernel. Which kernel a call
takes depends on all its sizes, so every test here asks for the plan and fails
if its call does not reach that kernel: small requests get there side by side
(copies of them that share blocks) or with loose bounds (a wide block table)."""
import math

import pytest
import torch

import attention_reference as ref
from attention_bounds import attention_seen
from test_gpu_kv_attention import filled
from test_gpu_kv_cache import ints, offsets_of

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("dit_rowwise_amax_b200")

OK, INDEX = 0, 6


def attend(q, cache, table, lens, offs, copies, width, frame, scale):
    """The batch `copies` times over, its block table `width` entries wide; q
    and out get rows behind the last request. Returns out and lse of the first
    copy; the others' are compared with them bit for bit."""
    n, t = offs[-1], cache[0].shape[2]
    wide = [row + [1 << 30] * (width - len(row)) for row in table] * copies
    all_offs = [c * n + o for c in range(copies) for o in offs[:-1]] + [copies * n]
    behind = torch.full((3,) + q.shape[1:], float("nan"), dtype=q.dtype, device=q.device)
    big = torch.cat([q[:n]] * copies + [behind])
    args = (big, cache, ints(wide), ints(lens * copies), ints(all_offs))
    most = max(b - a for a, b in zip(offs, offs[1:]))
    assert fp8.kv_cache_attention_plan(*args, max_q=most, max_kv=width * t)[0] == 256, "not the tcgen05 kernel"
    out = torch.full(big.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = fp8.kv_cache_attention(*args, max_q=most, max_kv=width * t, causal=frame, scale=scale, out=out, return_lse=True)
    torch.cuda.synchronize()
    assert bool((out[copies * n:] == 7.0).all()), "rows behind the last request were written"
    for c in range(1, copies):
        assert torch.equal(out[c * n: (c + 1) * n], out[:n]) and torch.equal(lse[c * n: (c + 1) * n], lse[:n]), "copies differ"
    return out[:n], lse[:n]


def sizes_for_tiles(heads, cache, table, lens, offs, how):
    """(copies, table width) that bring a call to the tcgen05 kernel."""
    t, kv = cache[0].shape[2], cache[0].shape[1]
    rows = max(b - a for a, b in zip(offs, offs[1:])) * (heads // kv)
    width, copies = max(len(r) for r in table), 1
    while copies * len(lens) * kv * -(-rows // 16) * (width * t + 384) <= 216000:
        if how == "loose":
            width = width * 2
        else:
            copies += 1
    return copies, width


def check(q, cache, table, lens, offs, frame=0, scale=None, how="copies"):
    dim = q.shape[2]
    copies, width = sizes_for_tiles(q.shape[1], cache, table, lens, offs, how)
    got, lse = attend(q, cache, table, lens, offs, copies, width, frame, scale)
    want, want_lse, bound, lse_bound = ref.attention(q, cache, table, lens, offs, dim ** -0.5 if scale is None else scale, frame)
    n = offs[-1]
    err = (got.double() - want)[:n].abs()
    assert not bool(err.isnan().any())
    assert bool((err <= bound[:n]).all()), f"worst error / bound {float((err / bound[:n].clamp(min=1e-300)).max()):.3f}"
    assert torch.equal(want_lse[:n].isinf(), lse.isinf())
    fin = ~want_lse[:n].isinf()
    d = (lse.double() - want_lse[:n])[fin].abs()
    assert bool((d <= lse_bound[:n][fin]).all()), f"lse off by {float(d.max())}"
    return got


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


HOW = ["copies", "loose"]  # the latter with ranges of keys
SHAPES = [(1, 1, 64, 16), (4, 4, 128, 32), (8, 1, 128, 64), (6, 2, 64, 128), (10, 2, 128, 128), (12, 1, 64, 16)]


def normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def table_for(lens, t, seed=0):
    need = [-(-n // t) for n in lens]
    pages = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
    return [[pages.pop() if j < n else -7 for j in range(max(need + [1]))] for n in need], sum(need) + 2


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("heads,kv,dim,t", SHAPES)
@pytest.mark.parametrize("new,lens", [([26], [900]), ([130, 2], [131, 257]), ([300], [300]), ([65, 257, 1], [0, 1000, 64])])
@pytest.mark.parametrize("frame", [0, 7])
def test_head_layouts_and_blocks(heads, kv, dim, t, new, lens, frame, how):
    g = torch.Generator("cuda").manual_seed(heads * 7 + dim + len(lens))
    table, blocks = table_for(lens, t)
    cache = filled(blocks, t, kv, dim, g)
    check(normal((sum(new), heads, dim), g), cache, table, lens, offsets_of(new), frame, how=how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [40, 200])
def test_more_new_tokens_than_cached_ones(dim, new, how):
    g = torch.Generator("cuda").manual_seed(new)
    cache = filled(4, 16, 2, dim, g)
    for n in (0, 1, 3):
        check(normal((new, 4, dim), g), cache, [[2, 1]], [n], [0, new], 1, how=how)


@pytest.mark.parametrize("how", HOW)
def test_strided_queries_and_outputs(how):
    """q out of a merged projection, an output with heads in between."""
    g = torch.Generator("cuda").manual_seed(2)
    new, heads, kv, dim, t, lens = 150, 4, 2, 128, 32, [70, 33]
    table, blocks = table_for(lens, t)
    cache = filled(blocks, t, kv, dim, g)
    offs = [0, new, new + 1]
    copies, width = sizes_for_tiles(heads, cache, table, lens, offs, how)
    n = copies * (new + 1)
    merged = normal((n + 6, (heads + 2 * kv) * dim), g)
    merged[n:] = float("nan")
    q = merged[:, : heads * dim].view(-1, heads, dim)
    q[: n] = q[: new + 1].repeat(copies, 1, 1)
    wide = torch.full((n + 6, heads + 3, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (q, cache, ints([row + [1 << 30] * (width - len(row)) for row in table] * copies), ints(lens * copies),
            ints([c * (new + 1) + o for c in range(copies) for o in (0, new)] + [n]))
    assert fp8.kv_cache_attention_plan(*args, max_q=new)[0] == 256
    out = fp8.kv_cache_attention(*args, max_q=new, out=wide[:, 1: 1 + heads])
    want, _, bound, _ = ref.attention(q[: new + 1], cache, table, lens, offs, dim ** -0.5, 0)
    for c in range(copies):
        assert bool(((out[c * (new + 1): (c + 1) * (new + 1)].double() - want).abs() <= bound).all())
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 1 + heads:] == 5).all()) and bool((wide[n:] == 5).all())


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new", [9, 140])
@pytest.mark.parametrize("exponent", [-118, -60, 5, 8, 20, 100])
def test_scales_over_the_whole_range(new, exponent, how):
    g = torch.Generator("cuda").manual_seed(4)
    heads, kv, dim, t, n = 2, 1, 64, 16, 150
    cache = filled(11, t, kv, dim, g)
    cache.v_scale.fill_(2.0 ** exponent)
    cache.v_scale[::2] *= 0.5
    table = [list(range(10, 0, -1))]
    q = normal((new, heads, dim), g)
    check(q, cache, table, [n], [0, new], how=how)
    cache.v_scale.fill_(1.0)
    cache.k_scale.fill_(2.0 ** exponent)
    e = max(-110, min(110, -9 - exponent))
    check((q.float() * 2.0 ** e).bfloat16(), cache, table, [n], [0, new], how=how)


@pytest.mark.parametrize("how", HOW)
def test_queries_up_to_the_largest_bf16(how):
    g = torch.Generator("cuda").manual_seed(5)
    new, heads, kv, dim, t, n = 140, 2, 1, 64, 16, 150
    cache = filled(10, t, kv, dim, g)
    cache.k_scale.fill_(2.0 ** -120)
    q = (torch.randn((new, heads, dim), generator=g, device="cuda") * 2.0 ** 124).bfloat16()
    q[:, 1, 5] = torch.finfo(torch.bfloat16).max
    q[:, 0, 7] = -torch.finfo(torch.bfloat16).max
    check(q, cache, [list(range(10))], [n], [0, new], scale=2.0 ** -14, how=how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new", [20, 300])
@pytest.mark.parametrize("order", [1, -1])
def test_value_scales_of_different_blocks(new, order, how):
    """V's unit grows step by step (order < 0), or is the first block's for all."""
    g = torch.Generator("cuda").manual_seed(6)
    heads, kv, dim, t, blocks = 4, 2, 128, 16, 52
    cache = filled(blocks, t, kv, dim, g)
    e = torch.arange(blocks, device="cuda") // 4
    e = e if order > 0 else 12 - e
    cache.v_scale.copy_(torch.exp2(-e.float())[:, None].expand(-1, kv))
    cache.k_scale.copy_(torch.exp2(-6.0 - (torch.arange(blocks, device="cuda") % 5).float())[:, None].expand(-1, kv))
    q, n = normal((new, heads, dim), g), blocks * t - 5
    check(q, cache, [list(range(blocks))], [n], [0, new], how=how)
    check(q, cache, [list(range(blocks))], [n], [0, new], 1, how=how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new", [40, 300])
def test_one_block_much_smaller_and_all_zero_blocks(new, how):
    g = torch.Generator("cuda").manual_seed(7)
    heads, kv, dim, t = 2, 1, 64, 32
    cache = filled(20, t, kv, dim, g)
    for b in (0, 3, 4, 19):
        cache.v[b] = 0
        cache.v_scale[b] = 2.0 ** -120
    cache.v_scale[7] = 2.0 ** -48
    check(normal((new, heads, dim), g), cache, [list(range(20))], [20 * t], [0, new], how=how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new", [17, 129, 300])
def test_scores_far_apart(new, how):
    """Rows whose maximum keeps rising by much, or is reached by one key only."""
    heads, kv, dim, t, n = 1, 1, 64, 16, 400
    cache = filled(25, t, kv, dim, torch.Generator("cuda").manual_seed(3))
    k = torch.zeros((n, 1, dim), device="cuda")
    k[:, 0, 0] = torch.arange(n, device="cuda") / 4.0
    k[200, 0, 1] = 100.0
    v = torch.randn((n, 1, dim), device="cuda")
    table = [list(range(25))]
    fp8.kv_cache_append(cache, k.bfloat16(), v.bfloat16(), ints(table), ints([n]), ints([0, n]), max_new=n)
    q = torch.zeros((new, heads, dim), device="cuda")
    q[:, 0, 0] = torch.linspace(-8, 8, new, device="cuda")
    q[::3, 0, 1] = 5.0
    check(q.bfloat16(), cache, table, [n], [0, new], 0, scale=1.0, how=how)
    check(q.bfloat16(), cache, table, [n], [0, new], 1, scale=1.0, how=how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new,heads,t", [(26, 4, 64), (200, 2, 64), (140, 2, 16)])
def test_unused_memory_may_hold_anything(new, heads, t, how):
    """NaN codes and NaN scales in blocks and rows that no query sees."""
    g = torch.Generator("cuda").manual_seed(8)
    dim, n = 128, t + 6
    cache = filled(5, t, 2, dim, g)
    used = [3, 1]
    for i in (0, 2, 4):
        cache.k[i] = 0x7F
        cache.v[i] = 0xFF
        cache.k_scale[i] = float("nan")
        cache.v_scale[i] = float("inf")
    cache.k[1, :, n - t:] = 0x7F
    cache.v[1, :, n - t:] = 0x7F
    q = normal((new, heads, dim), g)
    check(q, cache, [used + [0]], [n], [0, new], 0, how=how)
    check(q, cache, [used + [0]], [n], [0, new], 1, how=how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new,t", [(140, 32), (20, 16), (300, 128)])
def test_block_indices_out_of_range(new, t, how):
    """Tokens of a bad block are masked (NaN codes where its tile's buffers may
    hold them), the call goes on and reports."""
    g = torch.Generator("cuda").manual_seed(10)
    cache = filled(6, t, 1, 64, g)
    q, n = normal((new, 2, 64), g), 4 * t - 8
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        for table in ([[3, bad, 0, 5]], [[bad, 2, bad, bad]], [[bad] * 4]):
            check(q, cache, table, [n], [0, new], 0, how=how)
            assert fp8.device_error() == INDEX
    check(q, cache, [[3, 1, 0, 5]], [n], [0, new], 0, how=how)
    assert fp8.device_error() == OK


@pytest.mark.parametrize("how", HOW)
def test_lengths_out_of_range_leave_the_request_out(how):
    g = torch.Generator("cuda").manual_seed(11)
    new, t, cache = 140, 32, filled(6, 32, 1, 64, g)
    copies, width = sizes_for_tiles(2, cache, [[0, 1]], [60], [0, new], how)
    n = copies + 1
    q = normal((n * new, 2, 64), g)
    table = [[0, 1] + [1 << 30] * (width - 2)] * n
    want, _, bound, _ = ref.attention(q, cache, [[0, 1]] * n, [60] * n, offsets_of([new] * n), 0.125, 0)
    for at, length, offs in ((0, width * t + 1, None), (n - 1, -1, None), (0, 60, (0, -1)), (n - 1, 60, (n, n * new + 1))):
        lens, o = [60] * n, offsets_of([new] * n)
        lens[at] = length
        if offs is not None:
            o[offs[0]] = offs[1]
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        args = (q, cache, ints(table), ints(lens), ints(o))
        assert fp8.kv_cache_attention_plan(*args, max_q=2 * new)[0] == 256
        fp8.kv_cache_attention(*args, max_q=2 * new, out=out)
        assert fp8.device_error() == INDEX
        bad = torch.zeros(n * new, dtype=torch.bool, device="cuda")
        bad[at * new: (at + 1) * new] = True
        assert bool((out[bad] == 7.0).all())
        assert bool(((out.double() - want)[~bad].abs() <= bound[~bad]).all())


def test_cache_beyond_32_bit_offsets():
    """K and V of more than 2^32 bytes each; the blocks in use lie at the end."""
    g = torch.Generator("cuda").manual_seed(13)
    t, kv, dim, blocks, new = 128, 16, 128, 16500, 260
    cache = fp8.KVCache.empty(blocks, t, kv, dim)
    used = [16499, 16385, 16400, 3]
    part = filled(4, t, kv, dim, g)
    for i, p in enumerate(used):
        for a, b in zip(cache, part):
            a[p] = b[i]
    check(normal((new, kv, dim), g), cache, [used], [500], [0, new])


@pytest.mark.parametrize("new", [40, 150])
def test_calls_side_by_side_on_streams(new):
    """Eight calls on four streams at once, workspaces allocated per call."""
    g = torch.Generator("cuda").manual_seed(16)
    cache = filled(130, 32, 4, 64, g)
    pages = list(range(130))
    copies, width = sizes_for_tiles(8, cache, [pages], [4100], [0, new], "loose")
    tab, lens, offs = ints([pages + [-1] * (width - 130)]), ints([4100]), ints([0, new])
    qs = [normal((new, 8, 64), g) for _ in range(8)]
    assert fp8.kv_cache_attention_plan(qs[0], cache, tab, lens, offs, max_q=new)[0] == 256
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(4)], []
    for i, q in enumerate(qs):
        with torch.cuda.stream(streams[i % 4]):
            outs.append(fp8.kv_cache_attention(q, cache, tab, lens, offs, max_q=new, causal=i % 2))
    torch.cuda.synchronize()
    for i, (q, out) in enumerate(zip(qs, outs)):
        want, _, bound, _ = ref.attention(q, cache, [pages], [4100], [0, new], 0.125, i % 2)
        assert bool(((out.double() - want).abs() <= bound).all())
    assert fp8.device_error() == OK


def test_whole_video_over_itself():
    """Every token of a video sees every token: 32760 queries over 32760 keys;
    rows of all row tiles against the reference, a second run bit for bit."""
    g = torch.Generator("cuda").manual_seed(18)
    n, heads, dim, t = 32760, 2, 128, 128
    cache = filled(256, t, heads, dim, g)
    pages = torch.randperm(256, generator=torch.Generator().manual_seed(1)).tolist()
    q = normal((n, heads, dim), g)
    args = (q, cache, ints([pages]), ints([n]), ints([0, n]))
    assert fp8.kv_cache_attention_plan(*args, max_q=n)[0] == 256
    out = fp8.kv_cache_attention(*args, max_q=n)
    assert torch.equal(out, fp8.kv_cache_attention(*args, max_q=n))
    rows = torch.cat([torch.arange(0, n, 251), torch.tensor([127, 128, 255, 256, n - 1])])
    want, _, bound, _ = ref.attention(q[rows.cuda()], cache, [pages], [n], [0, len(rows)], dim ** -0.5, 0)
    assert bool(((out[rows.cuda()].double() - want).abs() <= bound).all())
    assert fp8.device_error() == OK


def check_seen(q, cache, pages, n, frame=0, scale=None, how="copies", **kw):
    """One request against attention_bounds.attention_seen."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    copies, width = sizes_for_tiles(q.shape[1], cache, [pages], [n], [0, q.shape[0]], how)
    got, lse = attend(q, cache, [pages], [n], [0, q.shape[0]], copies, width, frame, scale)
    want, want_lse, bound, lse_bound = attention_seen(q, cache, pages, n, frame, scale, **kw)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), f"worst error / bound {float((err / bound).max()):.3f}, NaN {bool(err.isnan().any())}"
    fin = ~want_lse.isinf()
    assert torch.equal(~fin, lse.isinf()) and bool(((lse.double() - want_lse).abs() <= lse_bound)[fin].all())


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("small,large", [(-120, 9), (-120, 40), (-100, 30), (40, -100)])
def test_slots_that_meet_value_scales_far_apart(small, large, how):
    """At most 128 rows: the two slots take the even and the odd tiles of 128
    keys, one of them with V far below the other's. First all rows see both,
    then some see only the first tile: what the other holds is not theirs."""
    g = torch.Generator("cuda").manual_seed(19)
    new, heads, dim, t, n = 100, 1, 64, 128, 200
    cache = filled(2, t, heads, dim, g)
    cache.v_scale[0], cache.v_scale[1] = 2.0 ** small, 2.0 ** large
    if small == -120:
        cache.v[0] = 0
    q = normal((new, heads, dim), g)
    check_seen(q, cache, [0, 1], n, how=how)
    check_seen(q, cache, [0, 1], n, 1, how=how)


def test_smallest_values_over_a_long_cache():
    """2^-112 on average over 12.6 million keys: 2^-120 over the softmax's sum
    is far below fp32's normal range."""
    requests, new, dim, t, n = 148, 20, 64, 128, 3 << 22
    cache = filled(1, t, 1, dim, torch.Generator("cuda").manual_seed(20))
    cache.v.fill_(0x78)  # 256
    cache.v_scale.fill_(2.0 ** -120)
    table = torch.zeros((requests, n // t), dtype=torch.int32, device="cuda")
    q = torch.zeros((requests * new, 1, dim), dtype=torch.bfloat16, device="cuda")
    args = (q, cache, table, ints([n] * requests), ints(offsets_of([new] * requests)))
    assert fp8.kv_cache_attention_plan(*args, max_q=new) == (256, 1)
    out, lse = fp8.kv_cache_attention(*args, max_q=new, return_lse=True)
    # Equal weights and values: every sum of up to 2^24 of either is exact.
    assert bool(((out.double() * 2.0 ** 112 - 1).abs() <= 2.0 ** -8 + 2.0 ** -20).all())
    assert bool(((lse.double() - math.log(n)).abs() <= 2.0 ** -20 * math.log(n)).all())
    assert fp8.device_error() == OK


@pytest.mark.parametrize("requests,new,kernel", [(2400, 1, 8), (148, 200, 256)])
def test_many_weights_far_below_the_largest(requests, new, kernel):
    """A million keys at 2^-27 of one key's weight make up 2^-7 of the whole;
    where that key's value is 0 they are all there is."""
    dim, t, n = 64, 128, 1 << 20
    cache = filled(2, t, 1, dim, torch.Generator("cuda").manual_seed(21))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(2.0 ** -8)
    cache.k.zero_()
    cache.k[:, :, :, 0] = 0xB8  # -1
    cache.v.fill_(0x78)         # 256
    cache.k[0, :, 0, 0] = 0     # the first block's first key: score 0, the others -27 (log2)
    cache.v[0, :, 0, ::2] = 0
    table = torch.ones((requests, n // t), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    q = torch.zeros((requests * new, 1, dim), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 27.0
    args = (q, cache, table, ints([n] * requests), ints(offsets_of([new] * requests)))
    assert fp8.kv_cache_attention_plan(*args, max_q=new) == (kernel, 1)
    out, lse = fp8.kv_cache_attention(*args, max_q=new, scale=math.log(2.0), return_lse=True)
    mass = (n - 1) * 2.0 ** -27
    # bf16 2^-8; a weight of 2^-20 is exact in fp16; the exponent -27 is off by
    # 27 2^-23 or less (fp32 scale and product), exp2 by 2^-22, running fp32 sums of
    # at most n / 64 terms by 2^-24 each.
    near = 2.0 ** -8 + 27 * 2.0 ** -23 + 2.0 ** -22 + n / 64 * 2.0 ** -24
    want = mass / (1 + mass)
    assert bool(((out[:, :, ::2].double() - want).abs() <= near * want).all()), float(out[0, 0, 0]) / want
    assert bool(((lse.double() - math.log1p(mass)).abs() <= n / 64 * 2.0 ** -24 + 2.0 ** -20).all())
    assert fp8.device_error() == OK


@pytest.mark.parametrize("new", [150, 300])
@pytest.mark.parametrize("apart", [25, 60, 200])
def test_blocks_that_the_mask_hides_do_not_count(new, apart):
    """The first rows see only blocks with V far below that of the blocks that
    the mask hides from them, some in the same 128 keys."""
    g = torch.Generator("cuda").manual_seed(22)
    heads, dim, t, n = 2, 64, 16, 330
    cache = filled(21, t, 1, dim, g)
    cache.v_scale.fill_(2.0 ** (100 - apart))
    cache.v_scale[7::3] = 2.0 ** 100
    check_seen(normal((new, heads, dim), g), cache, list(range(21)), n, 1, floor="contribution")


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new", [60, 300])
@pytest.mark.parametrize("apart", [20, 35, 90])
def test_rows_whose_weight_lies_on_a_small_block(new, apart, how):
    """One block's scores are 2^45 above the others', its V 2^apart below
    theirs: with 20 and 35 it still makes up the row."""
    g = torch.Generator("cuda").manual_seed(23)
    heads, dim, t, n = 1, 128, 32, 600
    cache = filled(19, t, heads, dim, g)
    cache.v_scale[6] = 2.0 ** (-8 - apart)
    q = normal((new, heads, dim), g)
    q[:, :, 0] = 4.0
    cache.k[:, :, :, 0] = 0
    cache.k_scale.fill_(2.0 ** -9)
    cache.k[6, :, :, 0] = 0x7E  # 448 2^-9 x 4 = 3.5
    scale = 45 * math.log(2.0) / 3.5
    cache.k[:, :, :, 1:] = cache.k[:, :, :, 1:] & 0x9F  # other products small beside that
    check_seen(q, cache, list(range(19)), n, scale=scale, how=how, floor="either" if how == "loose" else "contribution")


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("new,frame", [(40, 0), (128, 1), (300, 0), (300, 7)])
@pytest.mark.parametrize("dim,t", [(64, 16), (128, 32), (64, 128)])
def test_value_scales_anywhere(new, frame, dim, t, how):
    """Tiles with one unit first, then blocks whose V scales go up and down by
    anything up to 2^200, zeros and bad blocks among them."""
    g = torch.Generator("cuda").manual_seed(24)
    heads, n = 2, 11 * 128 - 3
    blocks = 11 * 128 // t
    cache = filled(blocks, t, 1, dim, g)
    e = torch.randint(-100, 100, (blocks,), generator=torch.Generator().manual_seed(new + dim))
    e[: 3 * 128 // t] = e[: 3 * 128 // t] % 12
    e[blocks // 2] = -120
    cache.v[blocks // 2] = 0
    cache.v_scale.copy_(torch.exp2(e.float())[:, None])
    pages = list(range(blocks))
    check_seen(normal((new, heads, dim), g), cache, pages, n, frame, how=how, floor="either")
    cache.v[blocks - 2], cache.k[blocks - 2] = 0xFF, 0x7F  # what a bad index may not reach
    check(normal((new, heads, dim), g), cache, [pages[: blocks - 2] + [-1, blocks - 1]], [n], [0, new], frame, how=how)
    assert fp8.device_error() == INDEX
