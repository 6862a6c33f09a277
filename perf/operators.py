"""The full-attention operators of a hybrid stack at a prefix-cache hit, as cases to be timed and compared.

Two operators, used in this order for every new token of a full-attention layer:

``norm_rope``
    RMS norm of every query and key head, the position rotation in the same pass, and the rotated keys and the
    values written to their slots of a paged cache.
``attention``
    attention of a chunk of new tokens (a suffix, a whole prompt, or one token) over the paged cache that already
    holds them: row i of a sequence with n new tokens and a context of L sees the keys 0 .. L - n + i, with a window
    only the last `window` of those.

``run`` computes them with elementary torch operations in 32 bits, or with the package's kernels where ``own`` is true.
Lengths and page layouts come from the case, values from the seed.
"""
import math
import random

import torch

own = False

NORM_EPS = 1e-6
BASE = 10000.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- cases

def _norm_rope(name, dtype, rows, heads, kv_heads, dim, rot, interleaved, page, far):
    case = {"op": "norm_rope", "dtype": dtype, "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "page": page, "far": far}
    return dict(case, name=name) if name else case


def _attention(name, dtype, heads, kv_heads, dim, page, batch, ctx, new, window, lse, layout):
    case = {"op": "attention", "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "batch": batch,
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1], "window": window, "lse": lse, "layout": layout}
    return dict(case, name=name) if name else case


def listed():
    return [
        # the first token after a hit, one request: latency alone counts
        _norm_rope("norm_rope one token", "bf16", 1, 16, 4, 128, 128, False, 16, 8192),
        # a decode step of 64 requests
        _norm_rope("norm_rope 64 tokens", "bf16", 64, 32, 8, 128, 128, False, 16, 32768),
        # fp32, odd sizes, a quarter-open rotation of neighbouring pairs
        _norm_rope("norm_rope f32 odd", "f32", 777, 6, 2, 64, 32, True, 48, 100000),
        # the 1024-token suffix of the 32-head stack behind its 32K prefix
        _norm_rope("norm_rope suffix", "bf16", 1024, 32, 32, 128, 128, False, 64, 32768),
        # all suffixes of the 64-request ragged batch at once
        _norm_rope("norm_rope ragged batch", "bf16", 67001, 16, 4, 128, 64, False, 32, 32768),
        # the first token after a hit: one request, 32K of context
        _attention("attention decode one", "bf16", 32, 8, 128, 16, 1, (32769, 32769), (1, 1), 0, False, 1),
        # a decode step of 64 ragged requests
        _attention("attention decode batch", "bf16", 16, 4, 128, 64, 64, (1024, 32768), (1, 1), 0, False, 2),
        # fp32, short odd chunks (a few drafted tokens each), scores' log-sums kept for a later merge
        _attention("attention f32 odd", "f32", 6, 2, 64, 48, 5, (77, 2001), (1, 33), 0, True, 3),
        # a sliding window with a group of 6 heads and pages that no tile boundary falls on
        _attention("attention window", "bf16", 24, 4, 64, 48, 8, (900, 16385), (100, 1000), 1024, True, 4),
        # the single layer: 512 new tokens behind 8K
        _attention("attention suffix 8K", "bf16", 16, 16, 128, 64, 1, (8704, 8704), (512, 512), 0, False, 5),
        # the stack's layer: 1024 new tokens behind 32K, no heads shared
        _attention("attention suffix 32K", "bf16", 32, 32, 128, 64, 1, (33792, 33792), (1024, 1024), 0, False, 6),
        # the 64-request ragged batch: suffixes of 64 to 2048 behind prefixes of 1K to 32K
        _attention("attention ragged batch", "bf16", 16, 4, 128, 32, 64, (3000, 34000), (64, 2048), 0, False, 7),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dim = rng.choice((64, 128, 128))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    kv_heads = rng.choice((1, 2, 4, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 4, 6, 7, 8))
    page = rng.choice((16, 16, 32, 48, 64, 128, 256))
    if rng.random() < 0.4:
        rows = _log_int(rng, 1, 60000 * 24 // (heads + 2 * kv_heads) if dtype == "bf16" else 20000)
        return _norm_rope(None, dtype, rows, heads, kv_heads, dim, rng.choice((16, 32, 64, dim, dim)), rng.random() < 0.3, page,
                          _log_int(rng, 1, 1000000))
    window = 0 if rng.random() < 0.7 else _log_int(rng, 16, 8192)
    while True:
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 34000)
        lo = rng.randint(max(1, hi // 16), hi)
        new = (1, 1) if rng.random() < 0.4 else (0 if batch > 2 else 1, _log_int(rng, 2, 2048))
        if rng.random() < 0.15:
            new = (hi, hi)  # whole prompts, nothing cached before
        case = _attention(None, dtype, heads, kv_heads, dim, page, batch, (lo, hi), new, window, rng.random() < 0.3, rng.randint(1, 10 ** 6))
        w = work(case)
        # fp32 runs on the CUDA cores: up to a 4096-token prompt's work there, the largest listed case's otherwise
        if w["flops"] <= (6e12 if dtype == "bf16" else 1e11) and w["bytes"] <= 2e9 and max(_lengths(case)[1], default=0) <= 34000:
            return case


def _lengths(case):
    """New tokens and contexts (new ones included) of each sequence, from the case alone."""
    r = random.Random(case["layout"])
    new, ctx = [], []
    for _ in range(case["batch"]):
        c = r.randint(case["ctx_lo"], case["ctx_hi"])
        new.append(min(c, r.randint(case["new_lo"], case["new_hi"])))
        ctx.append(c)
    if sum(new) == 0:
        new[0] = 1
    return new, ctx


def _visible(case):
    """Pairs of query row and visible key, and the keys that at least one row of their sequence sees, over all sequences."""
    pairs = keys = 0
    for n, c in zip(*_lengths(case)):
        if n == 0:
            continue
        w = case["window"] or c
        first = c - n + 1  # keys that the first row sees without a window
        full = max(0, min(n, w - first))  # rows that the window does not cut
        pairs += full * first + full * (full - 1) // 2 + (n - full) * w
        keys += min(c, n - 1 + w)
    return pairs, keys


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm_rope":
        per_row = 2 * (case["heads"] + 2 * case["kv_heads"]) * case["dim"] * size + 16
        flops = case["rows"] * (case["heads"] + case["kv_heads"]) * (4 * case["dim"] + 3 * case["rot"])
        return {"bytes": case["rows"] * per_row, "flops": flops}
    pairs, keys = _visible(case)
    rows = sum(_lengths(case)[0])
    wide = case["dim"] * size
    bytes_ = 2 * keys * case["kv_heads"] * wide + 2 * rows * case["heads"] * wide + 4 * keys // case["page"]
    return {"bytes": bytes_ + (4 * rows * case["heads"] if case["lse"] else 0), "flops": 4 * pairs * case["heads"] * case["dim"]}


# --------------------------------------------------------------------------------------------------------- inputs

def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    heads, kv, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    state = {"case": case}
    if case["op"] == "norm_rope":
        rows = case["rows"]
        pages = -(-rows // page) + 3
        # one projection's rows: q, k and v are slices of it
        qkv = _randn(g, (rows, heads + 2 * kv, dim), dtype)
        state["q"], state["k"], state["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        state["q_weight"] = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
        state["k_weight"] = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
        state["positions"] = case["far"] + torch.randint(0, 4096, (rows,), generator=g, device="cuda")
        state["inv_freq"] = BASE ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        state["k_cache"] = _randn(g, (pages, page, kv, dim), dtype)
        state["v_cache"] = _randn(g, (pages, page, kv, dim), dtype)
        # consecutive rows fill pages taken from a free list in no order; the last pages stay as they are
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(rows, device="cuda")
        state["slots"] = order[at // page] * page + at % page
        state["q_out"] = torch.empty((rows, heads, dim), dtype=dtype, device="cuda")
    else:
        new, ctx = _lengths(case)
        need = [-(-c // page) for c in ctx]
        pages = sum(need) + 2
        # normed heads times a learned weight's size: scores of about 2.5 standard deviations
        state["q"] = _randn(g, (sum(new), heads, dim), dtype, 2.5)
        state["k_cache"] = _randn(g, (pages, page, kv, dim), dtype)
        state["v_cache"] = _randn(g, (pages, page, kv, dim), dtype)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((len(ctx), max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        state["page_table"] = table
        state["new"], state["ctx"] = new, ctx
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        state["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        state["context_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        state["o"] = torch.zeros((sum(new), heads, dim), dtype=dtype, device="cuda")
        state["lse"] = torch.zeros((sum(new), heads), dtype=torch.float32, device="cuda") if case["lse"] else None
    if own:
        import gated_deltanet_state_tail_b200 as gdn
        state["gdn"] = gdn
        if case["op"] == "attention":
            state["attention"] = gdn.PagedAttention(heads, kv, dim, dtype, max_batch=case["batch"], max_rows=sum(state["new"]))
    return state


# ------------------------------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["op"] == "norm_rope":
        if own:
            state["gdn"].qk_norm_rope(
                state["q"], state["k"], state["positions"], state["inv_freq"], q_weight=state["q_weight"], k_weight=state["k_weight"],
                eps=NORM_EPS, interleaved=case["interleaved"], v=state["v"], k_cache=state["k_cache"], v_cache=state["v_cache"],
                slots=state["slots"], q_out=state["q_out"])
        else:
            _plain_norm_rope(state, case)
        return {"q": state["q_out"], "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    if own:
        state["attention"].run(state["q"], state["k_cache"], state["v_cache"], state["page_table"], state["cu_seqlens"],
                               state["context_len"], state["o"], lse_out=state["lse"], window=case["window"])
    else:
        _plain_attention(state, case)
    return {"o": state["o"], "lse": state["lse"]} if case["lse"] else {"o": state["o"]}


def _plain_norm_rope(state, case):
    rot, half = case["rot"], case["rot"] // 2
    # angles of far positions need 64 bits; their sines do not
    angle = torch.remainder(state["positions"].double()[:, None] * state["inv_freq"], 2 * math.pi).float()[:, None]
    cos, sin = torch.cos(angle), torch.sin(angle)

    def one(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * weight
        y = x.clone()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :half], x[..., half:rot]
            y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    state["q_out"].copy_(one(state["q"], state["q_weight"]))
    kv, dim = case["kv_heads"], case["dim"]
    state["k_cache"].view(-1, kv, dim)[state["slots"]] = one(state["k"], state["k_weight"]).to(state["k_cache"].dtype)
    state["v_cache"].view(-1, kv, dim)[state["slots"]] = state["v"]


def _plain_attention(state, case):
    heads, kv, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    scale = dim ** -0.5
    row = 0
    for b, (n, c) in enumerate(zip(state["new"], state["ctx"])):
        if n == 0:
            continue
        pages = state["page_table"][b, :-(-c // page)].long()
        k = state["k_cache"][pages].reshape(-1, kv, dim)[:c].permute(1, 0, 2)
        v = state["v_cache"][pages].reshape(-1, kv, dim)[:c].permute(1, 0, 2)
        q = state["q"][row:row + n].reshape(n, kv, heads // kv, dim).permute(1, 2, 0, 3)
        at = torch.arange(c - n, c, device="cuda")[:, None]
        key = torch.arange(c, device="cuda")
        hidden = key > at
        if case["window"]:
            hidden = hidden | (key <= at - case["window"])
        step = kv if heads * n * c <= 1 << 28 else 1  # key heads at a time
        for h in range(0, kv, step):
            s = torch.matmul(q[h:h + step].float().reshape(-1, heads // kv * n, dim), k[h:h + step].float().transpose(1, 2)) * scale
            s = s.view(-1, heads // kv, n, c).masked_fill_(hidden, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s.sub_(top))
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(-1, heads // kv * n, c), v[h:h + step].float()).view(-1, heads // kv, n, dim) / total
            a, z = h * (heads // kv), (h + step) * (heads // kv)
            state["o"][row:row + n, a:z] = o.reshape(z - a, n, dim).transpose(0, 1).to(state["o"].dtype)
            if state["lse"] is not None:
                state["lse"][row:row + n, a:z] = (top + torch.log(total)).reshape(z - a, n).t()
        row += n


# -------------------------------------------------------------------------------------------- from the definition

def exact(case, seed):
    """What run() returns, in 64 bits."""
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    return _exact_norm_rope(state, case) if case["op"] == "norm_rope" else _exact_attention(state, case)


def _exact_norm_rope(state, case):
    rot = case["rot"]

    def turned(x, weight):
        x = x.double()
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + NORM_EPS) * weight.double()
        # each pair as a complex number, turned by its angle
        pairs = x[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
        axis = -1 if case["interleaved"] else -2
        z = torch.complex(pairs.select(axis, 0).contiguous(), pairs.select(axis, 1).contiguous())
        z = z * torch.polar(torch.ones_like(angle), angle)
        return torch.cat([torch.stack([z.real, z.imag], axis).flatten(-2), x[..., rot:]], -1)

    angle = torch.outer(state["positions"].double(), state["inv_freq"])[:, None, :]
    k_cache, v_cache = state["k_cache"].double(), state["v_cache"].double()
    page, row = state["slots"] // case["page"], state["slots"] % case["page"]
    k_cache[page, row] = turned(state["k"], state["k_weight"])
    v_cache[page, row] = state["v"].double()
    return {"q": turned(state["q"], state["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attention(state, case):
    group, page = case["heads"] // case["kv_heads"], case["page"]
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(state["q"].shape[:2], dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, c) in enumerate(zip(state["new"], state["ctx"])):
        at = torch.arange(c, device="cuda")
        where, inside = state["page_table"][b][at // page].long(), at % page
        for first in range(0, n, 512):  # rows at a time
            rows = range(row + first, row + min(n, first + 512))
            last = torch.arange(c - n + first, c - n + first + len(rows), device="cuda")
            sees = at[None] <= last[:, None]
            if case["window"]:
                sees &= at[None] > last[:, None] - case["window"]
            for h in range(case["heads"]):
                if h % group == 0:
                    k, v = state["k_cache"][where, inside, h // group].double(), state["v_cache"][where, inside, h // group].double()
                s = torch.einsum("id,jd->ij", state["q"][rows.start:rows.stop, h].double(), k) / math.sqrt(case["dim"])
                s = torch.where(sees, s, torch.full_like(s, -math.inf))
                total = torch.logsumexp(s, -1)
                lse[rows.start:rows.stop, h] = total
                o[rows.start:rows.stop, h] = torch.einsum("ij,jd->id", torch.exp(s - total[:, None]), v)
        row += n
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
