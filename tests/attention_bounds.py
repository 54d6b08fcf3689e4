"""A float64 attention of one request and an error bound to which only the keys
that a row sees contribute, for calls whose blocks' scales lie far apart or
whose weights do."""
import math

import torch

import attention_reference as ref


def attention_seen(q, cache, pages, n, frame, scale, floor="weight"):
    """(out, lse, bound, lse_bound) of one request, q [new, heads, dim], its
    last tokens being the queries.

    With A = sum p |v| per element, over seen keys: p as fp16 is off by half a
    step, 2^-11 of it while normal, else by 2^-25 in units in which the largest
    p so far is at least 2^6 (2^7, but for what approximate references lose).
    So the floor is 2^-31 sum_t r_t 448 S_t, r_t the running maximum
    of p over the keys up to the end of t's 128 keys (a later, larger p scales
    the earlier error down with it), S_t the block's scale, which carries codes
    up to 448. Where the block scale is part of p's exponent (floor =
    "contribution") the running maximum of p S takes the place of r_t S_t;
    "either": whichever is larger, for calls that do both.
    A score is an fp32 sum of D products: off by at most (D + 4) 2^-24 scale
    sum |q k| plus D 2^-38 scale max |q| max |k| (q's own scaling); exp2 adds
    2^-22 and its argument's rounding, 2^-24 of the distance to the reference
    (at most twice the row's largest |score|, in log2 units, and V's exponent):
    relative, in numerator and denominator alike. The fp32 sums over the n keys
    add n 2^-24 each, bf16 rounding 2^-8 of the result."""
    k, v, ks, vs = cache
    t, dim, g = k.shape[2], k.shape[3], q.shape[1] // k.shape[1]
    values, idx = ref.e4m3_table(q.device), torch.tensor(pages[: -(-n // t)], dtype=torch.int64, device=q.device)
    limit = ref.key_limits(q.shape[0], n, frame, q.device)
    seen = torch.arange(n, device=q.device)[None] < limit[:, None]
    ends = torch.clamp((torch.arange(n, device=q.device) // 128 + 1) * 128, max=n) - 1
    outs = []
    for h in range(q.shape[1]):
        kk = (values[k[idx, h // g].long()] * ks[idx, h // g].double()[:, None, None]).reshape(-1, dim)[:n]
        vv = (values[v[idx, h // g].long()] * vs[idx, h // g].double()[:, None, None]).reshape(-1, dim)[:n]
        sv = vs[idx, h // g].double().repeat_interleave(t)[:n]
        x = q[:, h].double()
        s = torch.where(seen, x @ kk.T * scale, torch.full((), -math.inf, dtype=torch.float64, device=q.device))
        z = torch.logsumexp(s, 1)
        p = torch.where(seen, torch.exp(s - z.clamp(min=-1e300)[:, None]), torch.zeros_like(s))
        out, a = p @ vv, p @ vv.abs()

        def most(y):
            return torch.where(seen, y, torch.zeros_like(s)).amax(1)
        mass, top, expo = most(x.abs() @ kk.abs().T * scale), most(s.abs()), most(sv.log2().abs()[None].expand_as(s))
        e = (dim + 4) * 2.0 ** -24 * mass + 2.0 ** -22 + 2.0 ** -24 * (2 * 1.45 * top + expo)
        e = e + dim * 2.0 ** -38 * scale * x.abs().amax(1) * most(kk.abs().amax(1)[None].expand_as(s))
        weight, contribution = torch.cummax(p, 1).values[:, ends] * sv, torch.cummax(p * sv, 1).values[:, ends]
        run = {"weight": weight, "contribution": contribution, "either": torch.maximum(weight, contribution)}[floor]
        lost = 2.0 ** -31 * 448 * torch.where(seen, run, torch.zeros_like(s)).sum(1)
        bound = 1.01 * (2.0 ** -11 * a + 2.0 ** -8 * out.abs()) + (2 * e + 2 * n * 2.0 ** -24)[:, None] * a + lost[:, None] + 1e-44
        outs.append((out, z, bound, e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + z.abs().nan_to_num(posinf=0.0))))
    return [torch.stack(y, 1) for y in zip(*outs)]
