"""Appending to the E4M3 key / value cache: codes and scales have one right
answer and are compared bit for bit with the float64 reference."""
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("dit_rowwise_amax_b200")

OK, INDEX = 0, 6


def zeroed(*args):
    cache = fp8.KVCache.empty(*args)
    for x in cache:
        x.zero_()
    return cache


def make_table(lens, t, spare=2, seed=0):
    need = [-(-n // t) for n in lens]
    pages = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(need + [1])
    return [[pages.pop() if j < n else -7 for j in range(width)] for n in need], sum(need) + spare


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets_of(new):
    o = [0]
    for n in new:
        o.append(o[-1] + n)
    return o


def rand(shape, g, amp=True):
    x = torch.randn(shape, generator=g, device="cuda")
    if amp:
        x = x * torch.exp2(torch.randint(-12, 13, (shape[0], 1, 1), generator=g, device="cuda").float())
    return x.bfloat16()


def run_append(cache, k, v, table, lens, offs, **kw):
    want = [ref.append(cache[i].cpu(), cache[i + 2].cpu(), x.cpu(), table, lens, offs) for i, x in ((0, k), (1, v))]
    fp8.kv_cache_append(cache, k, v, ints(table), ints(lens), ints(offs), **kw)
    torch.cuda.synchronize()
    assert fp8.device_error() == OK
    for i in (0, 1):
        assert torch.equal(cache[i].cpu(), want[i][0])
        assert torch.equal(cache[i + 2].cpu(), want[i][1])


@pytest.mark.parametrize("t", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 3), (128, 2)])
@pytest.mark.parametrize("steps", [[(5, 1, 0, 130), (1, 1, 1, 1), (64, 0, 3, 16)], [(0, 17, 128, 129), (300, 1, 0, 1)]])
def test_append_steps(t, dim, heads, steps):
    """Requests of different lengths (none at all among them), step after step:
    blocks that start anew, fill up, grow their scale, end exactly full."""
    g = torch.Generator("cuda").manual_seed(t + dim)
    lens = [0] * 4
    final = [sum(s[i] for s in steps) for i in range(4)]
    table, blocks = make_table(final, t)
    cache = fp8.KVCache.empty(blocks, t, heads, dim)
    for x in cache:
        x.fill_(77)  # what an earlier user left behind
    for new in steps:
        lens = [a + b for a, b in zip(lens, new)]
        offs = offsets_of(new)
        run_append(cache, rand((offs[-1], heads, dim), g), rand((offs[-1], heads, dim), g), table, lens, offs, max_new=max(new))


def test_token_by_token_scale_growth():
    """One token at a time into one block, each larger than all before: the
    block's other codes, unused rows' too, come along at every step."""
    g = torch.Generator("cuda").manual_seed(1)
    cache = zeroed(3, 16, 2, 64)
    cache.k.copy_(torch.arange(16 * 64, device="cuda").view(16, 64) % 127)
    for i in range(16):
        k = (rand((1, 2, 64), g, False).float() * 2.0 ** (i / 2 - 4)).bfloat16()
        v = (rand((1, 2, 64), g, False).float() * 2.0 ** (-i)).bfloat16()
        run_append(cache, k, v, [[1]], [i + 1], [0, 1], max_new=1)


def special_rows():
    tiny, sub, top = 2.0 ** -126, 2.0 ** -133, 1.5 * 2.0 ** 127
    rows = [[0.0] * 64, [-0.0] * 64, [sub] * 64, [-tiny, 0.0] * 32, [top, -1.0] * 32, [448.0, -448.0, 447.0, 1e-3] * 16,
            [448.0 * 1.01, 17.0, 18.0, 19.0] * 16, [1.75, 1.7578125, 0.109375, 2.0 ** -9] * 16, [57344.0, 60000.0] * 32,
            [2.0 ** -112 * 1.75, 2.0 ** -113] * 32, [2.0 ** -111, 3.0 * 2.0 ** -121] * 32]
    return torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16).cuda()


def test_special_values_one_per_block():
    x = special_rows()[:, None, :]
    n = x.shape[0]
    cache = zeroed(n, 16, 1, 64)
    run_append(cache, x.contiguous(), x.flip(0).contiguous(), [[i] for i in range(n)], [1] * n, list(range(n + 1)), max_new=1)


def test_special_values_after_one_another():
    """Zero, subnormal and huge tokens in one block, one call and token by token."""
    x = special_rows()[:, None, :].contiguous()
    n = x.shape[0]
    cache = zeroed(2, 16, 1, 64)
    run_append(cache, x, x.flip(0).contiguous(), [[0]], [n], [0, n], max_new=n)
    for i in range(n):
        run_append(cache, x[i:i + 1], x[n - 1 - i:n - i], [[1]], [i + 1], [0, 1], max_new=1)


def test_merged_views_padded_rows_and_loose_bounds():
    """k and v as views of a merged projection; rows behind the last request
    are not read, blocks nobody reached keep every bit, max_new and the table
    are larger than needed."""
    g = torch.Generator("cuda").manual_seed(5)
    h, d, t, new = 2, 64, 32, [7, 40]
    offs = offsets_of(new)
    qkv = torch.randn((offs[-1] + 9, (4 + 2 * h) * d), generator=g, device="cuda").bfloat16()
    qkv[offs[-1]:] = float("nan")
    k, v = qkv[:, 4 * d: (4 + h) * d].view(-1, h, d), qkv[:, (4 + h) * d:].view(-1, h, d)
    cache = fp8.KVCache.empty(9, t, h, d)
    for x in cache:
        x.fill_(3)
    table = [[4, 99, -1, 8], [2, 7, 99, 99]]
    run_append(cache, k, v, table, [7, 40], offs, max_new=100)


def test_numbers_out_of_range_are_skipped_and_reported():
    h, d, t = 1, 64, 16
    k = torch.ones((8, h, d), dtype=torch.bfloat16, device="cuda")
    for table, lens, offs, most in (([[5]], [4], [0, 4], 4), ([[-1]], [4], [0, 4], 4), ([[0]], [17], [0, 4], 4),
                                    ([[0]], [2], [0, 4], 4), ([[0]], [4], [0, 9], 9), ([[0]], [4], [-1, 3], 4),
                                    ([[0]], [4], [4, 0], 4), ([[0]], [8], [0, 8], 4), ([[0]], [-1], [0, 0], 4)):
        cache = fp8.KVCache.empty(2, t, h, d)
        for x in cache:
            x.fill_(9)
        fp8.kv_cache_append(cache, k, k, ints(table), ints(lens), ints(offs), max_new=most)
        assert fp8.device_error() == INDEX
        assert fp8.device_error() == OK
        assert all(bool((x == 9).all()) for x in cache)


def test_graph_replay_reads_new_lengths():
    g = torch.Generator("cuda").manual_seed(3)
    h, d, t = 2, 128, 16
    table = [[3, 1, 0], [2, 5, 4]]
    cache = zeroed(6, t, h, d)
    k, v = rand((2, h, d), g), rand((2, h, d), g)
    tab, lens, offs = ints(table), ints([1, 1]), ints([0, 1, 2])
    mirror = [c.clone() for c in cache]
    fp8.kv_cache_append(mirror, k, v, tab, lens, offs, max_new=1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.kv_cache_append(cache, k, v, tab, lens, offs, max_new=1)
    want = [c.cpu().clone() for c in cache]
    for step in range(1, 35):
        k.copy_(rand((2, h, d), g))
        v.copy_(rand((2, h, d), g))
        n = [step, min(step, 20)]
        lens.copy_(ints(n))
        offs.copy_(ints([0, 1, 2] if step <= 20 else [0, 1, 1]))
        graph.replay()
        o = offs.tolist()
        for i, x in ((0, k), (1, v)):
            want[i], want[i + 2] = ref.append(want[i], want[i + 2], x.cpu(), table, n, o)
    torch.cuda.synchronize()
    assert fp8.device_error() == OK
    assert all(torch.equal(a.cpu(), b) for a, b in zip(cache, want))
