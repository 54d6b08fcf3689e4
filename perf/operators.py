"""The attention operators that follow the Q / K / V projections: rotary
positions with several axes, appending keys and values to an 8-bit cache with a
power-of-two scale for each block of tokens and head, and attention over that
cache.

``run`` computes them in plain torch operations, or, where ``own`` is true,
through the package's entry points. ``exact`` gives the same results from the
definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

FMAX = 448.0      # largest E4M3FN value
SCALE_MIN = -120  # smallest exponent of a block's scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One new token of each of 8 requests: a decoding step, latency counts.
        dict(name="rotary_tokens", op="rotary", tokens=8, q_heads=16, kv_heads=16, dim=128, axes="16,56,56", theta=256.0,
             halves=False, merged=False, fractional=False, first=40),
        # The whole video: 21 frames of 30 x 52 tokens, 16 heads of 128.
        dict(name="rotary_video", op="rotary", tokens=32760, q_heads=16, kv_heads=16, dim=128, axes="16,56,56", theta=256.0,
             halves=False, merged=False, fractional=False, first=0),
        # q and k as views of a merged projection, half-split pairs, shared key heads, a part of each head rotated,
        # stretched (fractional) positions far from the origin, an odd number of tokens.
        dict(name="rotary_merged", op="rotary", tokens=4099, q_heads=24, kv_heads=8, dim=128, axes="32,32,32", theta=10000.0,
             halves=True, merged=True, fractional=True, first=5000),
        # One new token of each of 64 requests into half-filled blocks.
        dict(name="append_tokens", op="append", requests=64, new_lo=1, new_hi=1, old_lo=10, old_hi=500, block=64, kv_heads=8, dim=128),
        # The keys and values of the whole video at once.
        dict(name="append_video", op="append", requests=1, new_lo=32760, new_hi=32760, old_lo=0, old_hi=0, block=128, kv_heads=16, dim=128),
        # Chunks of odd lengths behind odd lengths, small blocks, heads of 64.
        dict(name="append_ragged", op="append", requests=7, new_lo=1, new_hi=3001, old_lo=0, old_hi=777, block=16, kv_heads=12, dim=64),
        # One token over a short cache: latency.
        dict(name="attend_token", op="attention", requests=1, q_lo=1, q_hi=1, kv_lo=26, kv_hi=26, heads=16, kv_heads=16, dim=128,
             block=16, frame=0, lse=False),
        # A decoding batch: one token each, lengths from short to long, query heads in groups of four.
        dict(name="attend_batch", op="attention", requests=32, q_lo=1, q_hi=1, kv_lo=100, kv_hi=16001, heads=32, kv_heads=8, dim=128,
             block=64, frame=1, lse=False),
        # The 26 text tokens over the keys of the whole video.
        dict(name="attend_text", op="attention", requests=1, q_lo=26, q_hi=26, kv_lo=32760, kv_hi=32760, heads=16, kv_heads=16, dim=128,
             block=128, frame=0, lse=True),
        # One new frame of 1560 tokens over the cached video, itself included.
        dict(name="attend_frame", op="attention", requests=1, q_lo=1560, q_hi=1560, kv_lo=32760, kv_hi=32760, heads=16, kv_heads=16,
             dim=128, block=128, frame=0, lse=False),
        # Prompts of several requests behind cached ones: causal, shared key heads, heads of 64, odd lengths.
        dict(name="attend_prompts", op="attention", requests=5, q_lo=33, q_hi=2047, kv_lo=500, kv_hi=6001, heads=24, kv_heads=8, dim=64,
             block=32, frame=1, lse=True),
        # Four new frames at once, each seeing the frames up to its own.
        dict(name="attend_frames", op="attention", requests=1, q_lo=6240, q_hi=6240, kv_lo=32760, kv_hi=32760, heads=16, kv_heads=16,
             dim=128, block=128, frame=1560, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention"])
    if op == "rotary":
        dim = rng.choice([64, 96, 128, 128, 256])
        axes = {64: ["16,24,24", "32,32"], 96: ["32,32,32", "16,40,40", "64"], 128: ["16,56,56", "44,42,42", "32,32,32", "128"],
                256: ["64,96,96", "32,32"]}[dim]
        kv = rng.choice([1, 2, 4, 5, 8, 16])
        heads = kv * rng.choice([1, 1, 2, 3])
        tokens = _log(rng, 1, min(32760, 32760 * 32 * 128 // ((heads + kv) * dim)))
        return dict(op=op, tokens=tokens, q_heads=heads, kv_heads=kv, dim=dim, axes=rng.choice(axes), theta=rng.choice([256.0, 10000.0]),
                    halves=rng.random() < 0.5, merged=rng.random() < 0.5, fractional=rng.random() < 0.3, first=_log(rng, 1, 100000))
    if op == "append":
        dim, kv, block = rng.choice([64, 128]), rng.choice([1, 2, 3, 8, 12, 16]), rng.choice([16, 32, 64, 128])
        requests = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 32760 * 16 * 128 // (requests * kv * dim)))
        return dict(op=op, requests=requests, new_lo=rng.randint(1, hi), new_hi=hi, old_lo=0, old_hi=_log(rng, 1, 1000), block=block,
                    kv_heads=kv, dim=dim)
    dim, kv, block = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8, 16]), rng.choice([16, 32, 64, 128])
    heads = kv * rng.choice([1, 1, 2, 3, 4, 8])
    frame = rng.choice([0, 0, 1, 1, 390])
    requests = 1 if rng.random() < 0.4 else _log(rng, 1, 48)
    q_hi = 1 if rng.random() < 0.4 else _log(rng, 2, 4000)
    most = min(32760, 2.0e9 // (requests * heads * q_hi), 32760 * 16 * 128 * 2 // (requests * kv * dim))
    kv_hi = max(1, _log(rng, min(16, most), max(16, most)))
    q_hi = min(q_hi, kv_hi)
    return dict(op=op, requests=requests, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=rng.randint(1, kv_hi), kv_hi=kv_hi, heads=heads,
                kv_heads=kv, dim=dim, block=block, frame=frame, lse=rng.random() < 0.5)


def _lengths(case, lo, hi, n):
    """n whole numbers from lo to hi, the same for every seed; the last one is hi."""
    r = random.Random(1000003 * n + 1009 * hi + lo + case["block"])
    return [r.randint(lo, hi) for _ in range(n - 1)] + [hi]


def _sizes(case):
    """Per request: new tokens (queries) and the length of the cache with them."""
    if case["op"] == "append":
        new = _lengths(case, case["new_lo"], case["new_hi"], case["requests"])
        return new, [a + b for a, b in zip(new, _lengths(case, case["old_lo"], case["old_hi"], case["requests"]))]
    new = _lengths(case, case["q_lo"], case["q_hi"], case["requests"])
    return new, [max(a, b) for a, b in zip(new, _lengths(case, case["kv_lo"], case["kv_hi"], case["requests"]))]


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4.0 * n + 4.0 * case["tokens"] * len(case["axes"].split(",")), "flops": 3.0 * n}
    new, lens = _sizes(case)
    per_token = case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        touched = sum(-(-b // case["block"]) - (b - a) // case["block"] for a, b in zip(new, lens))
        return {"bytes": 2.0 * sum(new) * per_token * 3 + 2.0 * touched * case["kv_heads"] * 4, "flops": 2.0 * 3 * sum(new) * per_token}
    pairs = 0
    for a, b in zip(new, lens):
        if case["frame"]:
            pos = np.arange(b - a, b, dtype=np.int64)
            pairs += int(np.minimum(b, (pos // case["frame"] + 1) * case["frame"]).sum())
        else:
            pairs += a * b
    rows = sum(new) * case["heads"]
    blocks = sum(-(-b // case["block"]) for b in lens)
    return {"bytes": 2.0 * sum(lens) * per_token + 8.0 * blocks * case["kv_heads"] + 4.0 * blocks + 4.0 * rows * case["dim"]
            + (4.0 * rows if case["lse"] else 0.0), "flops": 4.0 * case["dim"] * case["heads"] * pairs}


# ----------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _filled_cache(g, blocks, kv_heads, block, dim):
    """Blocks of keys or values as an earlier append left them: codes and scales."""
    x = torch.randn((blocks, kv_heads, block, dim), generator=g, device="cuda").to(torch.bfloat16).float()
    x *= torch.exp2(torch.randint(-2, 3, (blocks, kv_heads, 1, 1), generator=g, device="cuda").float())
    scale = _block_scale(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "rotary":
        m, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        dims = tuple(int(a) for a in case["axes"].split(","))
        if case["merged"]:  # q, k and v side by side in one projection's output
            qkv = torch.randn((m, (hq + 2 * hk) * d), generator=g, device="cuda").to(torch.bfloat16)
            q, k = qkv[:, : hq * d].view(m, hq, d), qkv[:, hq * d: (hq + hk) * d].view(m, hk, d)
        else:
            q = torch.randn((m, hq, d), generator=g, device="cuda").to(torch.bfloat16)
            k = torch.randn((m, hk, d), generator=g, device="cuda").to(torch.bfloat16)
        at = case["first"] * 1560 + torch.arange(m, device="cuda")  # tokens of frames of 30 x 52
        grid = torch.stack([at // 1560, (at // 52) % 30, at % 52], 1)[:, : len(dims)]
        if len(dims) == 1:
            grid = at[:, None]
        pos = (grid.double() * 0.73).float() if case["fractional"] else grid.to(torch.int32)
        freqs = torch.cat([case["theta"] ** (-torch.arange(0, n, 2, dtype=torch.float64) / n) for n in dims])
        return dict(case=case, q=q, k=k, pos=pos.contiguous(), freqs=freqs, dims=dims, freqs_gpu=freqs.cuda(),
                    axis=torch.cat([torch.full((n // 2,), i) for i, n in enumerate(dims)]).cuda())
    new, lens = _sizes(case)
    t, hk, d = case["block"], case["kv_heads"], case["dim"]
    width = max(-(-n // t) for n in lens)
    need = [-(-n // t) for n in lens]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(int(seed))).tolist()
    table = [[order.pop() if j < n else 0 for j in range(width)] for n in need]
    kc, ks = _filled_cache(g, blocks, hk, t, d)
    vc, vs = _filled_cache(g, blocks, hk, t, d)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    state = dict(case=case, cache=(kc, vc, ks, vs), table=_ints(table), lens=_ints(lens), offsets=_ints(offsets), most=max(new),
                 longest=max(lens))
    if case["op"] == "append":
        amp = torch.exp2(torch.randint(-3, 4, (offsets[-1], 1, 1), generator=g, device="cuda").float())
        state["k"] = (amp * torch.randn((offsets[-1], hk, d), generator=g, device="cuda")).to(torch.bfloat16)
        state["v"] = torch.randn((offsets[-1], hk, d), generator=g, device="cuda").to(torch.bfloat16)
    else:
        state["q"] = torch.randn((offsets[-1], case["heads"], d), generator=g, device="cuda").to(torch.bfloat16)
        state["scale"] = 1.0 / math.sqrt(d)
    return state


# -------------------------------------------------------------- plain forms
def _block_scale(amax):
    """Smallest power of two S >= 2^-120 with amax <= 448 S."""
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa 2^exponent, mantissa in [0.5, 1)
    n = torch.where(amax > 0, exponent - 9 + (mantissa > FMAX / 512).to(exponent.dtype), torch.full_like(exponent, SCALE_MIN))
    return torch.ldexp(torch.ones_like(amax), n.clamp(min=SCALE_MIN))


def _rotate(x, cos, sin, halves):
    rot = 2 * cos.shape[1]
    y = x.float()
    a, b = (y[..., : rot // 2], y[..., rot // 2: rot]) if halves else (y[..., 0:rot:2], y[..., 1:rot:2])
    c, s = cos[:, None, :], sin[:, None, :]
    parts = [a * c - b * s, a * s + b * c]
    turned = torch.cat(parts, -1) if halves else torch.stack(parts, -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)


def _plain_rotary(s):
    angle = s["pos"].double()[:, s["axis"]] * s["freqs_gpu"]
    cos, sin = angle.cos().float(), angle.sin().float()
    return _rotate(s["q"], cos, sin, s["case"]["halves"]), _rotate(s["k"], cos, sin, s["case"]["halves"])


def _plain_append_one(x, codes, scale, s):
    """Writes the new tokens x into every block that they reach."""
    t = s["case"]["block"]
    new = s["offsets"].diff().long()
    first = s["lens"].long() - new
    request = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=x.shape[0])
    pos = torch.arange(x.shape[0], device="cuda") - s["offsets"][:-1].long()[request] + first[request]
    page, row = s["table"].long()[request, pos // t], pos % t
    # a block's old tokens: those in front of its request's first new one
    part = (first % t) > 0
    begun = s["table"].long().gather(1, (first // t).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    held = torch.zeros(codes.shape[0], dtype=torch.int32, device="cuda").index_add_(0, begun, part.int()) > 0
    touched = torch.zeros(codes.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.float().abs().amax(2), "amax")
    wanted = _block_scale(amax)
    after = torch.where(touched[:, None], torch.where(held[:, None], torch.maximum(scale, wanted), wanted), scale)
    again = torch.where(held & touched)[0]
    old = codes[again].view(torch.float8_e4m3fn).float() * (scale[again] / after[again])[:, :, None, None]
    codes[again] = old.to(torch.float8_e4m3fn).view(torch.uint8)
    value = (x.float() / after[page][:, :, None]).clamp(-FMAX, FMAX)
    codes[page, :, row] = value.to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(after)


def _plain_append(s):
    kc, vc, ks, vs = s["cache"]
    _plain_append_one(s["k"], kc, ks, s)
    _plain_append_one(s["v"], vc, vs, s)


def _plain_gather(codes, scale, table):
    """Every request's blocks one behind the other, in 32 bits: [requests, kv heads, tokens, dim]."""
    x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][:, :, :, None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attention(s):
    case, table = s["case"], s["table"].long()
    d, hk, g, frame = case["dim"], case["kv_heads"], case["heads"] // case["kv_heads"], case["frame"]
    new, lens = s["offsets"].diff().long(), s["lens"].long()
    total, b = s["q"].shape[0], len(new)
    request = torch.repeat_interleave(torch.arange(b, device="cuda"), new, output_size=total)
    at = torch.arange(total, device="cuda") - s["offsets"][:-1].long()[request]
    q = torch.zeros((b, s["most"], case["heads"], d), device="cuda")
    q[request, at] = s["q"].float() * s["scale"]
    q = q.view(b, s["most"], hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, s["most"] * g, d)
    keys, values = (_plain_gather(c, a, table) for c, a in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
    scores = q @ keys.transpose(2, 3)
    limit = lens[:, None].expand(b, s["most"])
    if frame:
        pos = lens[:, None] - new[:, None] + torch.arange(s["most"], device="cuda")
        limit = torch.minimum(limit, (pos // frame + 1) * frame)
    hidden = torch.arange(scores.shape[3], device="cuda") >= limit.repeat_interleave(g, 1)[:, None, :, None]
    scores.masked_fill_(hidden, float("-inf"))
    top = scores.amax(3, keepdim=True)
    p = scores.sub_(top).exp_()
    total_p = p.sum(3, keepdim=True)
    out = (p @ values) / total_p
    out = out.view(b, hk, s["most"], g, d).permute(0, 2, 1, 3, 4)[request, at].reshape(total, case["heads"], d).to(torch.bfloat16)
    if not case["lse"]:
        return out
    lse = (top + total_p.log())[..., 0].view(b, hk, s["most"], g).permute(0, 2, 1, 3)[request, at].reshape(total, case["heads"])
    return out, lse


# --------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    if own:
        import dit_rowwise_amax_b200 as fp8
        if case["op"] == "rotary":
            return fp8.rotary_axes(state["q"], state["k"], state["pos"], state["freqs"], state["dims"], interleaved=not case["halves"])
        if case["op"] == "append":
            fp8.kv_cache_append(state["cache"], state["k"], state["v"], state["table"], state["lens"], state["offsets"],
                                max_new=state["most"])
        else:
            return fp8.kv_cache_attention(state["q"], state["cache"], state["table"], state["lens"], state["offsets"],
                                          max_q=state["most"], max_kv=state["longest"], scale=state["scale"], causal=case["frame"],
                                          return_lse=case["lse"])
    elif case["op"] == "rotary":
        return _plain_rotary(state)
    elif case["op"] == "append":
        _plain_append(state)
    else:
        return _plain_attention(state)
    kc, vc, ks, vs = state["cache"]  # codes as the values that they stand for, and the blocks' scales
    return kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs


# ------------------------------------------------------------------- exact
def _exact_rotary(s):
    dims, outs = s["dims"], []
    for x in (s["q"], s["k"]):
        x, y, pair = x.double(), x.double().clone(), 0
        half = sum(dims) // 2
        for axis, n in enumerate(dims):
            for i in range(n // 2):
                angle = s["pos"][:, axis].double() * float(s["freqs"][pair])
                c, v = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
                lo, hi = (pair, pair + half) if s["case"]["halves"] else (2 * pair, 2 * pair + 1)
                y[:, :, lo] = x[:, :, lo] * c - x[:, :, hi] * v
                y[:, :, hi] = x[:, :, lo] * v + x[:, :, hi] * c
                pair += 1
        outs.append(y)
    return tuple(outs)


def _nearest_e4m3(x):
    """The nearest E4M3FN value of |x| <= 448, ties to the even mantissa, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _e4m3_values():
    table = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        table.append(-v if c & 128 else v)
    return torch.tensor(table, dtype=torch.float64, device="cuda")


def _exact_append(s):
    t, table = s["case"]["block"], s["table"].cpu().numpy()
    offsets, lens = s["offsets"].tolist(), s["lens"].tolist()
    value = _e4m3_values()
    outs = []
    for x, codes, scale in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        values, scales, x = value[codes.long()], scale.double().clone(), x.double()
        for r, n in enumerate(lens):
            start = n - (offsets[r + 1] - offsets[r])
            for j in range(start // t, -(-n // t)):
                lo, hi, page = max(start, j * t), min(n, (j + 1) * t), int(table[r, j])
                part = x[offsets[r] + lo - start: offsets[r] + hi - start].transpose(0, 1)  # [heads, tokens, dim]
                amax = part.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / 448.0)).clamp(min=-120.0)
                e = torch.where(torch.exp2(e) * 448.0 < amax, e + 1, e)
                e = torch.where((torch.exp2(e - 1) * 448.0 >= amax) & (e > -120), e - 1, e)
                to = torch.exp2(e)
                if lo > j * t:
                    to = torch.maximum(to, scales[page])
                    values[page] = _nearest_e4m3(values[page] * (scales[page] / to)[:, None, None])
                values[page, :, lo - j * t: hi - j * t] = _nearest_e4m3(part / to[:, None, None])
                scales[page] = to
        outs.append((values, scales))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _exact_attention(s):
    case, value = s["case"], _e4m3_values()
    g, frame, d, t = case["heads"] // case["kv_heads"], case["frame"], case["dim"], case["block"]
    offsets, lens = s["offsets"].tolist(), s["lens"].tolist()
    out = torch.zeros((offsets[-1], case["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((offsets[-1], case["heads"]), dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        a, b = offsets[r], offsets[r + 1]
        pages = s["table"][r, : -(-n // t)].long()
        limit = torch.full((b - a,), n, device="cuda")
        if frame:
            limit = torch.minimum(limit, ((n - (b - a) + torch.arange(b - a, device="cuda")) // frame + 1) * frame)
        seen = torch.arange(n, device="cuda")[None, :] < limit[:, None]
        for h in range(case["kv_heads"]):
            key, val = ((value[c[pages, h].long()] * z[pages, h].double()[:, None, None]).reshape(-1, d)[:n]
                        for c, z in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
            for i in range(h * g, (h + 1) * g):
                x = (s["q"][a:b, i].double() @ key.T) * s["scale"]
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                lse[a:b, i] = torch.logsumexp(x, 1)
                out[a:b, i] = torch.exp(x - lse[a:b, i, None]) @ val
    return (out, lse) if case["lse"] else out


def exact(case, seed):
    state = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "attention": _exact_attention}[case["op"]](state)
