"""Plain 64-bit forms of the full-attention operators, and bounds on what their kernels may be off by.

The bounds count roundings: a stored value is off by at most half a step, u(t) = finfo(t).eps / 2 of it; fp32 sums
of n terms by n u(f32) of the sum of the terms' sizes (twice that on the tensor cores, whose adders may truncate).
"""
import math

import torch

U32 = torch.finfo(torch.float32).eps / 2


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm_rope(x, positions, inv_freq, weight, eps, interleaved):
    """(y, bound) of [rows, heads, d] in 64 bits; the bound is for results computed in fp32 and rounded to x's type."""
    rows, heads, d = x.shape
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    out, size = y.clone(), y.abs()
    if rot:
        angle = positions.double()[:, None] * inv_freq[None]
        cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        i = torch.arange(rot // 2, device=x.device)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., first], y[..., second]
        out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
        size[..., first] = size[..., second] = a.abs() + b.abs()
    # mean of squares: at most d / 8 + 6 adds a lane and a tree; square root, two products and the rotation: 8 more
    # roundings; the sine and cosine: 4 steps (their argument, rounded to fp32, moves them by up to 3.2 of it); the
    # reference's own angle: far positions times 2^-52
    far = float(positions.abs().max()) * 2.0 ** -50 if rot and rows else 0.0
    fp32 = ((d / 8 + 6) / 2 + 12 + 2) * U32 + far
    return out, fp32 * size + half_step(x.dtype) * (out.abs() + fp32 * size)


def gather(cache, table, ctx):
    """Rows 0 .. ctx - 1 of one sequence: [ctx, Hkv, d]."""
    page = cache.shape[1]
    at = torch.arange(ctx, device=cache.device)
    return cache[table[at // page].long(), at % page]


def attention(q, k_cache, v_cache, page_table, cu, ctx, scale, window):
    """Per sequence (rows, o, o_bound, lse, lse_bound) in 64 bits."""
    heads, kv = q.shape[1], k_cache.shape[2]
    group, d = heads // kv, q.shape[2]
    dtype = q.dtype
    for b, c in enumerate(ctx):
        r0, r1 = cu[b], cu[b + 1]
        n = r1 - r0
        if n == 0:
            continue
        dev = q.device
        k = gather(k_cache, page_table[b], c).double().repeat_interleave(group, 1)
        v = gather(v_cache, page_table[b], c).double().repeat_interleave(group, 1)
        x = q[r0:r1].double()
        pos = torch.arange(n, device=dev)[:, None] + c - n
        key = torch.arange(c, device=dev)[None]
        sees = key <= pos
        if window:
            sees &= key > pos - window
        s = torch.einsum("nhd,jhd->hnj", x, k) * scale
        s = s.masked_fill(~sees, -math.inf)
        sizes = (torch.einsum("nhd,jhd->hnj", x.abs(), k.abs()) * scale).masked_fill(~sees, 0.0)
        lse = torch.logsumexp(s, -1) if c else torch.full((heads, n), -math.inf, dtype=torch.float64, device=dev)
        p = torch.exp(s - lse.clamp_min(-1e300)[..., None]).masked_fill(~sees, 0.0)
        o = torch.einsum("hnj,jhd->nhd", p, v)
        spread = torch.einsum("hnj,jhd->nhd", p, v.abs())
        top = sizes.amax(-1) if c else torch.zeros((heads, n), dtype=torch.float64, device=dev)
        adds = 2 if dtype == torch.bfloat16 else 1
        # a score: d products and sums, the scaling and the difference to the maximum, and what exp2 adds
        delta = (adds * (d + 8) * U32 * top + 16 * U32).t()[..., None]
        seen = sees.sum(-1).double()[:, None, None]
        sums = adds * (seen + 16) * U32
        weights = half_step(dtype) if dtype == torch.bfloat16 else 0.0   # p itself is rounded for the second product
        o_bound = (weights + 2 * delta + 2 * sums) * spread
        o_bound = o_bound + half_step(dtype) * (o.abs() + o_bound) + 1e-30
        lse_bound = (delta + sums)[..., 0] + 4 * U32 * lse.t().abs().nan_to_num(posinf=0.0) + 1e-30
        yield (r0, r1), o, o_bound, lse.t(), lse_bound


class Paged:
    """A paged cache with shuffled pages; everything outside the contexts holds NaN."""

    def __init__(self, ctx, kv, d, page, dtype, seed, layout="packed", k_scale=1.0, width=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        need = [-(-c // page) for c in ctx]
        self.pages = sum(need) + 3
        shape = (self.pages, page, kv, d)
        if layout == "packed":
            self.k = torch.full(shape, math.nan, dtype=dtype, device="cuda")
            self.v = torch.full(shape, math.nan, dtype=dtype, device="cuda")
        elif layout == "heads first":
            self.k = torch.full((self.pages, kv, page, d), math.nan, dtype=dtype, device="cuda").transpose(1, 2)
            self.v = torch.full((self.pages, kv, page, d), math.nan, dtype=dtype, device="cuda").transpose(1, 2)
        else:   # keys and values of a page in one buffer
            both = torch.full((self.pages, 2, page, kv, d), math.nan, dtype=dtype, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        order = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)
        # entries that no context needs point nowhere
        self.table = torch.full((len(ctx), width or max(1, max(need))), 2 ** 30, dtype=torch.int32, device="cuda")
        at = 0
        for b, (n, c) in enumerate(zip(need, ctx)):
            mine = order[at:at + n]
            self.table[b, :n] = mine
            at += n
            i = torch.arange(c, device="cuda")
            self.k[mine[i // page].long(), i % page] = (torch.randn((c, kv, d), generator=g, device="cuda") * k_scale).to(dtype)
            self.v[mine[i // page].long(), i % page] = torch.randn((c, kv, d), generator=g, device="cuda").to(dtype)
