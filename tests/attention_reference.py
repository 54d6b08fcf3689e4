"""Plain float64 forms of the rotary, cache and attention operators, from their
definitions, for tests."""
import math

import torch


def e4m3_table(device="cpu"):
    t = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        t.append(-v if c & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device=device)


def encode_e4m3(x):
    """Nearest E4M3FN codes of float64 x, ties to even, saturating; -0 kept."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    e = (e - 1).clamp(min=-6)
    steps = torch.round(torch.ldexp(a, 3 - e))  # mantissa in units of 2^(e - 3): 0 .. 16
    up = steps >= 16
    e, steps = torch.where(up, e + 1, e), torch.where(up, steps / 2, steps)
    code = torch.where(steps >= 8, (e + 7) * 8 + steps.to(e.dtype) - 8, steps.to(e.dtype))
    return (code.to(torch.int64) | (torch.signbit(x).to(torch.int64) << 7)).to(torch.uint8)


def scale_of(amax):
    """2^n, smallest n >= -120 with amax <= 448 2^n (amax a float)."""
    n = -120
    if amax > 0:
        n = max(-120, math.ceil(math.log2(amax / 448.0)) - 2)
        while math.ldexp(448.0, n) < amax:
            n += 1
    return math.ldexp(1.0, n)


def rotary(x, positions, freqs, axis_dims, interleaved):
    """x [M, H, D] -> float64, positions [M, axes], freqs float64 [R / 2]."""
    y = x.double().clone()
    axis = torch.cat([torch.full((n // 2,), i, dtype=torch.int64) for i, n in enumerate(axis_dims)]).to(x.device)
    angle = positions.double()[:, axis] * freqs.to(x.device)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    p = freqs.numel()
    a, b = (slice(0, 2 * p, 2), slice(1, 2 * p, 2)) if interleaved else (slice(0, p), slice(p, 2 * p))
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a] = xa * c - xb * s
    y[..., b] = xa * s + xb * c
    return y


def append(codes, scale, x, table, kv_lens, offsets):
    """New codes and scales after the append of x [total, heads, D] (all CPU)."""
    codes, scale = codes.clone(), scale.clone().double()
    t, values = codes.shape[2], e4m3_table()
    assert not bool(((codes & 127) == 127).any()), "NaN codes: no reference"
    for b, n in enumerate(kv_lens):
        start = n - (offsets[b + 1] - offsets[b])
        for j in range(start // t, -(-n // t) if n > start else 0):
            lo, hi, page = max(start, j * t), min(n, (j + 1) * t), table[b][j]
            for h in range(codes.shape[1]):
                part = x[offsets[b] + lo - start: offsets[b] + hi - start, h].double()
                s = scale_of(float(part.abs().max()))
                held = lo - j * t
                if held:
                    old = float(scale[page, h])
                    s = max(s, old)
                    if s != old:
                        codes[page, h] = encode_e4m3(values[codes[page, h].long()] * (old / s))
                codes[page, h, held: hi - j * t] = encode_e4m3(part / s)
                scale[page, h] = s
    return codes, scale.float()


def key_limits(n_new, kv_len, frame, device="cpu"):
    pos = kv_len - n_new + torch.arange(n_new, dtype=torch.int64, device=device)
    if not frame:
        return torch.full_like(pos, kv_len)
    return torch.where(pos < 0, torch.zeros_like(pos), torch.clamp((pos // frame + 1) * frame, max=kv_len))


def attention(q, cache, table, kv_lens, offsets, scale, frame, good_page=None):
    """float64 (out, lse, bound) of every request's rows; rows of no request are
    NaN. bound: largest error that the operator's roundings allow per element.

    With A = sum p |v| per element: rounding p to fp16 is off by half a step,
    2^-11 relative where p is a normal fp16, else by 2^-25 in units in which
    the row's largest p (tensor cores) or largest p times block scale (few
    rows) is at least 1; so the sum is off by at most 2^-11 A + 2^-25 n 448
    max(p S) + 2^-25 n max(p) 448 max(S). V on the tensor cores is an fp16 in
    units of the largest block scale: off by 2^-25 max(S). The output's
    rounding to bf16 adds 2^-8 |out|.
    A score is an fp32 sum of D products, off by at most (D + 4) 2^-24 scale
    sum |q k| =: e (D additions, the products' own and two scalings; q's own
    scaling to fp16 keeps all its bits down to 2^-38 of the row's largest:
    D 2^-38 max |q| max |k| more), plus the 2^-22 of an approximate exp2, its
    argument's rounding (2^-24 of a score relative to the row's reference, |s -
    m| <= 2 max |s|, in log2 units, and of the block scale's exponent added to
    it): each p is off by that relatively, numerator and denominator alike,
    hence twice; the fp32 sums over n keys add n 2^-24 each."""
    k, v, ks, vs = cache
    t, dim = k.shape[2], k.shape[3]
    g = q.shape[1] // k.shape[1]
    values = e4m3_table(q.device)
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse_bound = torch.zeros_like(lse)
    for b, n in enumerate(kv_lens):
        lo, hi = offsets[b], offsets[b + 1]
        pages = [table[b][j] for j in range(-(-n // t))]
        ok = torch.tensor([0 <= p < k.shape[0] for p in pages], dtype=torch.bool, device=q.device).repeat_interleave(t)[:n]
        idx = torch.tensor([p if 0 <= p < k.shape[0] else 0 for p in pages], dtype=torch.int64, device=q.device)
        limit = key_limits(hi - lo, n, frame, q.device)
        seen = (torch.arange(n, device=q.device)[None] < limit[:, None]) & ok[None]
        for h in range(q.shape[1]):
            kk = (values[k[idx, h // g].long()] * ks[idx, h // g].double()[:, None, None]).reshape(-1, dim)[:n]
            vv = (values[v[idx, h // g].long()] * vs[idx, h // g].double()[:, None, None]).reshape(-1, dim)[:n]
            x = q[lo:hi, h].double()
            s = torch.where(seen, x @ kk.T * scale, torch.full((1, 1), -math.inf, dtype=torch.float64, device=q.device))
            z = torch.logsumexp(s, 1) if n else torch.full((hi - lo,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.where(seen, torch.exp(s - z.clamp(min=-1e300)[:, None]), torch.zeros_like(s))
            out[lo:hi, h] = p @ vv
            lse[lo:hi, h] = z
            if n:
                mass = torch.where(seen, x.abs() @ kk.abs().T * scale, torch.zeros_like(s)).amax(1)
                top = torch.where(seen, s.abs(), torch.zeros_like(s)).amax(1)
                sv = vs[idx, h // g].double().repeat_interleave(t)[:n]
                expo = sv.log2().abs().max()
                e = (dim + 4) * 2.0 ** -24 * mass + 2.0 ** -22 + 2.0 ** -24 * (2 * 1.45 * top + expo)
                e = e + dim * 2.0 ** -38 * x.abs().amax(1) * kk.abs().max() * scale
                a = p @ vv.abs()
                floor = 2.0 ** -25 * (n * 448 * ((p * sv).amax(1) + p.amax(1) * sv.max()) + sv.max())
                bound[lo:hi, h] = (2.0 ** -11 * a + 2.0 ** -8 * out[lo:hi, h].abs()) * 1.01 \
                    + (2 * e + 2 * n * 2.0 ** -24)[:, None] * a + floor[:, None] + 1e-38
                lse_bound[lo:hi, h] = e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + z.abs().nan_to_num(posinf=0.0))
    return out, lse, bound, lse_bound
