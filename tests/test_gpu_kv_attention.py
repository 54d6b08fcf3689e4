"""Attention over the E4M3 cache against the float64 softmax of what the cache
holds, elementwise within the bound that the operator's roundings allow
(attention_reference.attention derives it)."""
import math
import random

import pytest
import torch

import attention_reference as ref
from test_gpu_kv_cache import ints, make_table, offsets_of, run_append, zeroed

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("dit_rowwise_amax_b200")

OK, INDEX = 0, 6


def filled(blocks, t, heads, dim, g, spread=2):
    """A cache of random codes (every finite code occurs) and scales."""
    k = torch.randint(0, 256, (blocks, heads, t, dim), generator=g, device="cuda", dtype=torch.int32)
    k = torch.where((k & 127) == 127, k - 1, k).to(torch.uint8)
    x = torch.randn((blocks, heads, t, dim), generator=g, device="cuda")
    v = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    # code sizes vary over seven octaves: keep keys' products near one
    ks = torch.exp2(torch.randint(-9, -9 + spread, (blocks, heads), generator=g, device="cuda").float())
    vs = torch.exp2(torch.randint(-8, -8 + spread, (blocks, heads), generator=g, device="cuda").float())
    return fp8.KVCache(k, v, ks, vs)


def check(q, cache, table, lens, offs, frame=0, scale=None, rows_behind=0, **kw):
    dim = q.shape[2]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = fp8.kv_cache_attention(q, cache, ints(table), ints(lens), ints(offs), causal=frame, scale=scale, out=out,
                                      return_lse=True, **kw)
    torch.cuda.synchronize()
    assert got is out
    want, want_lse, bound, lse_bound = ref.attention(q, cache, table, lens, offs, dim ** -0.5 if scale is None else scale, frame)
    n = offs[-1]
    assert bool((got[n:] == 7.0).all()), "rows behind the last request were written"
    err = (got.double() - want)[:n].abs()
    assert not bool(err.isnan().any())
    worst = float((err / bound[:n].clamp(min=1e-300)).max()) if n else 0.0
    assert bool((err <= bound[:n]).all()), f"worst error / bound {worst:.3f}"
    same_inf = want_lse[:n].isinf() == lse[:n].isinf()
    assert bool(same_inf.all())
    fin = ~want_lse[:n].isinf()
    d = (lse[:n].double() - want_lse[:n])[fin].abs()
    assert bool((d <= lse_bound[:n][fin]).all()), f"lse off by {float(d.max())}"
    return got


SHAPES = [  # heads, kv heads, dim, block
    (1, 1, 64, 16), (4, 4, 128, 32), (8, 1, 128, 64), (6, 2, 64, 128), (10, 2, 128, 128), (12, 1, 64, 16),
]


@pytest.mark.parametrize("heads,kv,dim,t", SHAPES)
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [26]), ([1, 1, 1], [1, 17, 300]), ([1, 0, 1], [129, 5, 0]), ([1], [2900]),
    ([3, 1, 8], [3, 16, 500]), ([26], [900]), ([130, 2], [131, 257]), ([300], [300]), ([65, 257, 1], [0, 1000, 64]),
])
@pytest.mark.parametrize("frame", [0, 1, 7])
def test_attention(heads, kv, dim, t, new, lens, frame):
    g = torch.Generator("cuda").manual_seed(heads * 7 + dim + len(lens))
    table, blocks = make_table(lens, t)
    cache = filled(blocks, t, kv, dim, g)
    offs = offsets_of(new)
    q = torch.randn((offs[-1], heads, dim), generator=g, device="cuda").bfloat16()
    check(q, cache, table, lens, offs, frame, max_q=max(new))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 5, 40, 200])
def test_more_new_tokens_than_cached_ones(dim, new):
    """Under a causal mask the first queries see nothing: 0 and -inf."""
    g = torch.Generator("cuda").manual_seed(new)
    cache = filled(4, 16, 2, dim, g)
    q = torch.randn((new, 4, dim), generator=g, device="cuda").bfloat16()
    for n in (0, 1, 3):
        check(q, cache, [[2, 1]], [n], [0, new], 1, max_q=new)


@pytest.mark.parametrize("new", [2, 150])
def test_strides_padding_and_loose_bounds(new):
    """q out of a merged projection, a strided output, rows behind the last
    request left alone, bounds larger than needed, garbage in unused entries."""
    g = torch.Generator("cuda").manual_seed(2)
    heads, kv, dim, t = 4, 2, 128, 32
    lens, offs = [70, 33], [0, new, new + 1]
    table, blocks = make_table(lens, t)
    table = [row + [1 << 30] * 3 for row in table]
    cache = filled(blocks, t, kv, dim, g)
    merged = torch.randn((new + 6, (heads + 2 * kv) * dim), generator=g, device="cuda").bfloat16()
    merged[new + 1:] = float("nan")
    q = merged[:, : heads * dim].view(-1, heads, dim)
    check(q, cache, table, lens, offs, 0, max_q=new + 100)
    wide = torch.full((new + 6, heads + 3, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    out = fp8.kv_cache_attention(q, cache, ints(table), ints(lens), ints(offs), max_q=new, out=wide[:, 1: 1 + heads])
    want, _, bound, _ = ref.attention(q, cache, table, lens, offs, dim ** -0.5, 0)
    assert bool(((out.double() - want)[: new + 1].abs() <= bound[: new + 1]).all())
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 1 + heads:] == 5).all()) and bool((wide[new + 1:] == 5).all())


@pytest.mark.parametrize("new", [1, 9, 140])
@pytest.mark.parametrize("exponent", [-118, -60, 5, 7, 8, 20, 100])
def test_scales_over_the_whole_range(new, exponent):
    """V of any size comes back in that size; K's is undone by the softmax scale."""
    g = torch.Generator("cuda").manual_seed(4)
    heads, kv, dim, t, n = 2, 1, 64, 16, 150
    cache = filled(11, t, kv, dim, g)
    cache.v_scale.fill_(2.0 ** exponent)
    cache.v_scale[::2] *= 0.5
    table = [list(range(10, 0, -1))]
    q = torch.randn((new, heads, dim), generator=g, device="cuda").bfloat16()
    check(q, cache, table, [n], [0, new], 0, max_q=new)
    if exponent <= 100:  # |K| to 2^109, q to 2^-98 or so: products near one
        cache.v_scale.fill_(1.0)
        cache.k_scale.fill_(2.0 ** exponent)
        e = max(-110, min(110, -9 - exponent))
        check((q.float() * 2.0 ** e).bfloat16(), cache, table, [n], [0, new], 0, max_q=new)


@pytest.mark.parametrize("new", [1, 9, 140])
def test_queries_up_to_the_largest_bf16(new):
    """Keys of blocks with the smallest scale bring them back near one."""
    g = torch.Generator("cuda").manual_seed(5)
    heads, kv, dim, t, n = 2, 1, 64, 16, 150
    cache = filled(10, t, kv, dim, g)
    cache.k_scale.fill_(2.0 ** -120)
    q = (torch.randn((new, heads, dim), generator=g, device="cuda") * 2.0 ** 124).bfloat16()
    q[:, 1, 5] = torch.finfo(torch.bfloat16).max
    q[:, 0, 7] = -torch.finfo(torch.bfloat16).max
    check(q, cache, [list(range(10))], [n], [0, new], 0, scale=2.0 ** -14, max_q=new)


@pytest.mark.parametrize("new", [1, 20, 300])
@pytest.mark.parametrize("order", [1, -1])
def test_value_scales_of_different_blocks(new, order):
    """V blocks whose scales rise or fall by 2^-12 in all, met in either order:
    every block keeps its own precision (tensor cores: exact to 2^-15 of the
    largest), keys' scales likewise."""
    g = torch.Generator("cuda").manual_seed(6)
    heads, kv, dim, t = 4, 2, 128, 16
    blocks = 52
    cache = filled(blocks, t, kv, dim, g)
    e = torch.arange(blocks, device="cuda") // 4
    e = e if order > 0 else 12 - e
    cache.v_scale.copy_(torch.exp2(-e.float())[:, None].expand(-1, kv))
    cache.k_scale.copy_(torch.exp2(-6.0 - (torch.arange(blocks, device="cuda") % 5).float())[:, None].expand(-1, kv))
    q = torch.randn((new, heads, dim), generator=g, device="cuda").bfloat16()
    n = blocks * t - 5
    check(q, cache, [list(range(blocks))], [n], [0, new], 0, max_q=new)
    check(q, cache, [list(range(blocks))], [n], [0, new], 1, max_q=new)


@pytest.mark.parametrize("new", [1, 40, 300])
def test_one_block_much_smaller_and_all_zero_blocks(new):
    """Blocks of zeros carry the smallest scale (2^-120) and weigh as any other;
    a block 2^-40 below the others adds nothing visible."""
    g = torch.Generator("cuda").manual_seed(7)
    heads, kv, dim, t = 2, 1, 64, 32
    cache = filled(20, t, kv, dim, g)
    for b in (0, 3, 4, 19):
        cache.v[b] = 0
        cache.v_scale[b] = 2.0 ** -120
    cache.v_scale[7] = 2.0 ** -48
    q = torch.randn((new, heads, dim), generator=g, device="cuda").bfloat16()
    check(q, cache, [list(range(20))], [20 * t], [0, new], 0, max_q=new)


@pytest.mark.parametrize("new", [1, 16, 129])
def test_scores_far_apart(new):
    """Rows whose maximum keeps rising by much, or is reached by one key only."""
    heads, kv, dim, t, n = 1, 1, 64, 16, 400
    cache = zeroed(25, t, kv, dim)
    k = torch.zeros((n, 1, dim), device="cuda")
    k[:, 0, 0] = torch.arange(n, device="cuda") / 4.0
    k[200, 0, 1] = 100.0
    v = torch.randn((n, 1, dim), device="cuda")
    table = [list(range(25))]
    run_append(cache, k.bfloat16(), v.bfloat16(), table, [n], [0, n], max_new=n)
    q = torch.zeros((new, 1, dim), device="cuda")
    q[:, 0, 0] = torch.linspace(-8, 8, new, device="cuda") if new > 1 else 8.0
    q[::3, 0, 1] = 5.0
    check(q.bfloat16(), cache, table, [n], [0, new], 0, max_q=new, scale=1.0)
    check(q.bfloat16(), cache, table, [n], [0, new], 1, max_q=new, scale=1.0)


@pytest.mark.parametrize("new,heads", [(1, 4), (26, 4), (200, 2)])
def test_unused_memory_may_hold_anything(new, heads):
    """NaN codes and NaN scales in blocks and rows that no query sees."""
    g = torch.Generator("cuda").manual_seed(8)
    dim, t, n = 128, 64, 70
    cache = filled(5, t, 2, dim, g)
    used = [3, 1]
    for i in range(5):
        if i not in used:
            cache.k[i] = 0x7F
            cache.v[i] = 0xFF
            cache.k_scale[i] = float("nan")
            cache.v_scale[i] = float("inf")
    cache.k[1, :, n - 64:] = 0x7F
    cache.v[1, :, n - 64:] = 0x7F
    q = torch.randn((new, heads, dim), generator=g, device="cuda").bfloat16()
    check(q, cache, [used + [0]], [n], [0, new], 0, max_q=new)
    check(q, cache, [used + [0]], [n], [0, new], 1, max_q=new)


@pytest.mark.parametrize("new", [1, 140])
def test_shared_blocks_and_split_ranges(new):
    """Two requests read the same prefix blocks; long caches are cut into
    ranges whose results join."""
    g = torch.Generator("cuda").manual_seed(9)
    heads, kv, dim, t = 4, 2, 128, 16
    cache = filled(300, t, kv, dim, g)
    a = list(range(299, 49, -1))
    b = a[:200] + list(range(0, 50))
    lens, offs = [4000 - 3, 3999], [0, new, 2 * new]
    q = torch.randn((2 * new, heads, dim), generator=g, device="cuda").bfloat16()
    check(q, cache, [a, b], lens, offs, 0, max_q=new)
    check(q, cache, [a, b], lens, offs, 390, max_q=new)
    one = fp8.kv_cache_attention(q, cache, ints([a, b]), ints(lens), ints(offs), max_q=new)
    two = fp8.kv_cache_attention(q, cache, ints([a, b]), ints(lens), ints(offs), max_q=new)
    assert torch.equal(one, two), "two runs differ"


@pytest.mark.parametrize("new", [1, 140])
def test_block_indices_out_of_range(new):
    """Tokens of a bad block are masked, the call goes on and reports."""
    g = torch.Generator("cuda").manual_seed(10)
    cache = filled(6, 32, 1, 64, g)
    q = torch.randn((new, 2, 64), generator=g, device="cuda").bfloat16()
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        table = [[3, bad, 0, 5]]
        check(q, cache, table, [120], [0, new], 0, max_q=new)
        assert fp8.device_error() == INDEX
    check(q, cache, [[3, 1, 0, 5]], [120], [0, new], 0, max_q=new)
    assert fp8.device_error() == OK


@pytest.mark.parametrize("new", [1, 140])
def test_lengths_out_of_range_leave_the_request_out(new):
    g = torch.Generator("cuda").manual_seed(11)
    cache = filled(6, 32, 1, 64, g)
    q = torch.randn((2 * new, 2, 64), generator=g, device="cuda").bfloat16()
    table = [[0, 1], [2, 3]]
    want, _, bound, _ = ref.attention(q, cache, table, [60, 60], [0, new, 2 * new], 0.125, 0)
    for lens, offs, most in (([65, 60], [0, new, 2 * new], new), ([-1, 60], [0, new, 2 * new], new),
                             ([60, 60], [-1, new, 2 * new], 2 * new), ([60, 60], [0, new, 2 * new + 1], 2 * new)):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        fp8.kv_cache_attention(q, cache, ints(table), ints(lens), ints(offs), max_q=most, out=out)
        assert fp8.device_error() == INDEX
        bad = slice(new, 2 * new) if offs[2] > 2 * new else slice(0, new)
        good = slice(0, new) if offs[2] > 2 * new else slice(new, 2 * new)
        assert bool((out[bad] == 7.0).all())
        assert bool(((out.double() - want)[good].abs() <= bound[good]).all())


def test_graphs_replay_with_new_lengths_side_by_side():
    """Two captured graphs with workspaces of their own run on two streams at
    once; a replay reads the lengths of its day."""
    g = torch.Generator("cuda").manual_seed(12)
    heads, kv, dim, t = 4, 1, 128, 64
    cache = filled(70, t, kv, dim, g)
    table = [list(range(0, 66))]
    cases = []
    for new in (1, 200):
        q = torch.randn((new, heads, dim), generator=g, device="cuda").bfloat16()
        lens, offs, out = ints([4200]), ints([0, new]), torch.empty_like(q)
        fp8.kv_cache_attention(q, cache, ints(table), lens, offs, max_q=new, out=out)
        s, graph, tab = torch.cuda.Stream(), torch.cuda.CUDAGraph(), ints(table)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            fp8.kv_cache_attention(q, cache, tab, lens, offs, max_q=new, out=out)
        cases.append((new, q, lens, out, s, graph, tab, offs))
    for n in (4200, 1, 999, 4224):
        for _, _, lens, _, _, _, _, _ in cases:
            lens.fill_(n)
        torch.cuda.synchronize()
        for _ in range(3):
            for _, _, _, _, s, graph, _, _ in cases:
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for new, q, _, out, _, _, _, _ in cases:
            want, _, bound, _ = ref.attention(q, cache, table, [n], [0, new], dim ** -0.5, 0)
            assert bool(((out.double() - want).abs() <= bound).all())
    assert fp8.device_error() == OK


@pytest.mark.parametrize("new", [1, 130])
def test_cache_beyond_32_bit_offsets(new):
    """K and V of more than 2^32 bytes each; the blocks in use lie at the end."""
    t, kv, dim, blocks = 128, 16, 128, 16500
    cache = fp8.KVCache.empty(blocks, t, kv, dim)
    used = [16499, 16385, 16400, 3]
    g = torch.Generator("cuda").manual_seed(13)
    part = filled(4, t, kv, dim, g)
    for i, p in enumerate(used):
        for a, b in zip(cache, part):
            a[p] = b[i]
    x = torch.randn((300, kv, dim), generator=g, device="cuda").bfloat16()
    q = torch.randn((new, kv, dim), generator=g, device="cuda").bfloat16()
    small = fp8.KVCache(*(c.clone() for c in part))
    for c, tab in ((cache, [used]), (small, [[0, 1, 2, 3]])):
        fp8.kv_cache_append(c, x, x, ints(tab), ints([500]), ints([0, 300]), max_new=300)
    a = fp8.kv_cache_attention(q, cache, ints([used]), ints([500]), ints([0, new]), max_q=new)
    b = fp8.kv_cache_attention(q, small, ints([[0, 1, 2, 3]]), ints([500]), ints([0, new]), max_q=new)
    assert torch.equal(a, b)
    assert all(torch.equal(c[p], s[i]) for c, s in zip(cache, small) for i, p in enumerate(used))
    check(q, small, [[0, 1, 2, 3]], [500], [0, new], 0, max_q=new)


def test_projection_rotary_append_attention():
    """A block's attention as it is used: Q / K / V projections sharing one
    quantised activation, rotary positions over (time, height, width), append,
    attention; a prompt, then frames, then single tokens, two requests."""
    hidden, heads, dim, t, dims = 256, 4, 64, 32, (16, 24, 24)
    g = torch.Generator("cuda").manual_seed(14)
    layers = [fp8.FP8Linear.from_weight((torch.randn((heads * dim, hidden), generator=g, device="cuda") * 0.06).bfloat16())
              for _ in range(3)]
    freqs = fp8.rotary_frequencies(dims, 256.0)
    steps = [(37, 12), (60, 60), (1, 1), (1, 0), (1, 1)]
    final = [sum(s[i] for s in steps) for i in range(2)]
    table, blocks = make_table(final, t)
    cache = zeroed(blocks, t, heads, dim)
    mirror = [c.cpu().clone() for c in cache]
    lens = [0, 0]
    for new in steps:
        lens = [a + b for a, b in zip(lens, new)]
        offs = offsets_of(new)
        x = torch.randn((offs[-1], hidden), generator=g, device="cuda").bfloat16()
        q, k, v = (y.view(-1, heads, dim) for y in fp8.scaled_linear_multi(layers, x))
        at = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).cuda()
        pos = torch.stack([at // 60, at % 60 // 10, at % 10], 1).int()
        q0, k0 = q.clone(), k.clone()
        q, k = fp8.rotary_axes(q, k, pos, freqs, dims, q_out=q, k_out=k)
        for got, x0 in ((q, q0), (k, k0)):
            want = ref.rotary(x0, pos, freqs, dims, True)
            assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * x0.double().abs().amax()).all())
        fp8.kv_cache_append(cache, k, v, ints(table), ints(lens), ints(offs), max_new=max(new))
        for i, y in ((0, k), (1, v)):
            mirror[i], mirror[i + 2] = ref.append(mirror[i], mirror[i + 2], y.cpu(), table, lens, offs)
            used = [p for row, n in zip(table, lens) for p in row[: -(-n // t)]]
            assert torch.equal(cache[i + 2].cpu()[used], mirror[i + 2][used])
            for b, n in enumerate(lens):
                for j in range(-(-n // t)):
                    m = min(t, n - j * t)
                    assert torch.equal(cache[i].cpu()[table[b][j], :, :m], mirror[i][table[b][j], :, :m])
        check(q, cache, table, lens, offs, 60, max_q=max(new))
    assert fp8.device_error() == OK


@pytest.mark.parametrize("new", [1, 12, 150])
def test_calls_side_by_side_on_streams(new):
    """Eight calls on four streams at once, workspaces allocated per call."""
    g = torch.Generator("cuda").manual_seed(16)
    cache = filled(130, 32, 2, 64, g)
    table, tab, lens, offs = [list(range(130))], ints([list(range(130))]), ints([4100]), ints([0, new])
    qs = [torch.randn((new, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(8)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(4)], []
    for i, q in enumerate(qs):
        with torch.cuda.stream(streams[i % 4]):
            outs.append(fp8.kv_cache_attention(q, cache, tab, lens, offs, max_q=new, causal=i % 2))
    torch.cuda.synchronize()
    for i, (q, out) in enumerate(zip(qs, outs)):
        want, _, bound, _ = ref.attention(q, cache, table, [4100], [0, new], 0.125, i % 2)
        assert bool(((out.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("new", [40, 300])
def test_split_ranges_under_a_causal_mask_with_empty_rows(new):
    """Ranges that no row of a tile sees, and rows that see nothing at all."""
    g = torch.Generator("cuda").manual_seed(17)
    cache = filled(70, 64, 1, 128, g)
    q = torch.randn((2 * new, 2, 128), generator=g, device="cuda").bfloat16()
    table = [list(range(66)), list(range(66))]
    check(q, cache, table, [4200, new - 7], [0, new, 2 * new], 1, max_q=new)
    check(q, cache, table, [4200, new - 7], [0, new, 2 * new], 2000, max_q=new)


@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    """Seeded draws over block sizes, head layouts, ragged and empty requests,
    masks and both kernels; every call twice, bit for bit the same."""
    r = random.Random(seed)
    for _ in range(6):
        dim, t, kv, g = r.choice([64, 128]), r.choice([16, 32, 64, 128]), r.choice([1, 2, 3]), r.choice([1, 2, 3, 8])
        n = r.choice([1, 1, 2, 5, 40])
        most_new, most_kv = r.choice([1, 2, 17, 40, 130, 260, 700] if n < 40 else [1, 3, 20]), r.choice([30, 200, 900, 3001])
        new, lens = [r.randint(0, most_new) for _ in range(n)], [r.randint(0, most_kv) for _ in range(n)]
        frame = r.choice([0, 0, 1, 13, 390])
        gen = torch.Generator("cuda").manual_seed(r.randrange(1 << 30))
        table, blocks = make_table(lens, t, seed=seed)
        cache = filled(blocks, t, kv, dim, gen, spread=r.choice([1, 4]))
        offs = offsets_of(new)
        q = torch.randn((offs[-1] + 3, kv * g, dim), generator=gen, device="cuda").bfloat16()
        q[offs[-1]:] = float("nan")
        first = check(q, cache, table, lens, offs, frame, max_q=max(new + [1])).clone()
        assert torch.equal(first, check(q, cache, table, lens, offs, frame, max_q=max(new + [1])))
    assert fp8.device_error() == OK


def test_other_stream():
    g = torch.Generator("cuda").manual_seed(15)
    cache = filled(20, 16, 2, 64, g)
    q = torch.randn((3, 4, 64), generator=g, device="cuda").bfloat16()
    table, tab, lens, offs = [list(range(20))], ints([list(range(20))]), ints([300]), ints([0, 3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = fp8.kv_cache_attention(q, cache, tab, lens, offs, max_q=3)
    s.synchronize()
    want, _, bound, _ = ref.attention(q, cache, table, [300], [0, 3], 0.125, 0)
    assert bool(((out.double() - want).abs() <= bound).all())
    assert math.isfinite(float(out.float().sum()))
