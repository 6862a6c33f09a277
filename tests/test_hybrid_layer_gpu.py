"""The full-attention operators as a hybrid stack uses them: the prefix is appended in chunks, the suffix and then
single tokens attend over it, beside the GDN layers' own prefill and decode of the same tokens."""
import pytest
import torch

import gated_deltanet_state_tail_b200 as gdn
import hybrid_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefix_suffix_and_decode(dtype):
    heads, kv, d, page, window = 8, 2, 128, 16, 0
    lens = [333, 70, 129]            # prefix of each request
    suffix = [40, 130, 1]
    steps = 3
    total = [p + s + steps for p, s in zip(lens, suffix)]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    qw, kw = torch.full((d,), 1.5, device="cuda"), torch.full((d,), 1.2, device="cuda")
    raw = [torch.randn((t, heads + 2 * kv, d), generator=g, device="cuda").to(dtype) for t in total]
    need = [-(-t // page) for t in total]
    order = torch.randperm(sum(need) + 1, generator=g, device="cuda")
    table = torch.zeros((3, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kc = torch.full((sum(need) + 1, page, kv, d), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    attn = gdn.PagedAttention(heads, kv, d, dtype, max_batch=3)
    i32 = dict(dtype=torch.int32, device="cuda")

    def step(begin, end):
        """Tokens begin[b] .. end[b] of every request through both operators."""
        rows = torch.cat([r[a:z] for r, a, z in zip(raw, begin, end)])
        pos = torch.cat([torch.arange(a, z, device="cuda") for a, z in zip(begin, end)])
        seq = torch.cat([torch.full((z - a,), b, device="cuda") for b, (a, z) in enumerate(zip(begin, end))])
        slots = table[seq, pos // page].long() * page + pos % page
        q, _ = gdn.qk_norm_rope(rows[:, :heads], rows[:, heads:heads + kv], pos, inv, qw, kw, v=rows[:, heads + kv:],
                                k_cache=kc, v_cache=vc, slots=slots)
        cu = torch.tensor([0] + [z - a for a, z in zip(begin, end)]).cumsum(0).to(**i32)
        o = torch.empty(q.shape, dtype=dtype, device="cuda")
        attn.run(q, kc, vc, table, cu, torch.tensor(end, **i32), o, window=window)
        attn.check()
        want = list(ref.attention(q, kc, vc, table, cu.tolist(), list(end), d ** -0.5, window))
        for (r0, r1), w, bound, _, _ in want:
            assert bool(((o[r0:r1].double() - w).abs() <= bound).all())
        return o

    step([0, 0, 0], [200, 70, 100])
    step([200, 70, 100], [333, 70, 129])            # the second request has nothing new
    step(lens, [p + s for p, s in zip(lens, suffix)])
    for i in range(steps):
        begin = [p + s + i for p, s in zip(lens, suffix)]
        step(begin, [x + 1 for x in begin])
    # the cache holds the whole sequences, rotated: against one norm + rotation of each in 64 bits
    for b, t in enumerate(total):
        pos = torch.arange(t, device="cuda")
        want, bound = ref.norm_rope(raw[b][:, heads:heads + kv], pos, inv, kw, 1e-6, False)
        assert bool(((ref.gather(kc, table[b], t).double() - want).abs() <= bound).all())
        assert torch.equal(ref.gather(vc, table[b], t), raw[b][:, heads + kv:])


def test_bench_hybrid_workload():
    """The bench's own run of the full-attention layers, one layer of them."""
    import types

    import bench
    line, = bench.bench_hybrid(types.SimpleNamespace(layers=3, steps=3, warmup=3))
    assert line["layers"] == 1 and line["value"] > 0
    for part in ("suffix", "decode"):
        assert 0 < line[part]["attention_roofline"]["frac"] < 1.5 and 0 < line[part]["norm_rope_ms"] < line["value"]


def test_beside_gdn_layers_on_another_stream():
    """A GDN prefill on one stream and paged attention on another give what each gives alone."""
    from gated_deltanet_state_tail_b200 import inputs
    t = inputs.draw_tensors(4096, 16, 128, 128, "bf16", 0.9, 0.999, 1, device="cuda")
    plan = gdn.PrefillPlan(16, 128, 128, "bf16", [0, 1024, 2048, 3000, 4096])
    o_gdn, st = torch.empty_like(t["v"]), torch.empty((4, 16, 128, 128), device="cuda")
    ctx, new = [5000, 700], [300, 1]
    cache = ref.Paged(ctx, 2, 128, 64, torch.bfloat16, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((301, 8, 128), generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (cache.k, cache.v, cache.table, torch.tensor([0, 300, 301], **i32), torch.tensor(ctx, **i32))
    attn = gdn.PagedAttention(8, 2, 128, "bf16", max_batch=2)
    o = torch.empty_like(q)
    attn.run(q, *args, o)
    plan.run(t["q"], t["k"], t["v"], t["alpha"], t["beta"], o_gdn, state_out=st)
    torch.cuda.synchronize()
    want, want_gdn, want_st = o.clone(), o_gdn.clone(), st.clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        plan.run(t["q"], t["k"], t["v"], t["alpha"], t["beta"], o_gdn, state_out=st, stream=a)
        attn.run(q, *args, o, stream=b)
    torch.cuda.synchronize()
    assert attn.status() == gdn.GDN_OK and plan.status() == gdn.GDN_OK
    assert torch.equal(o, want) and torch.equal(o_gdn, want_gdn) and torch.equal(st, want_st)
    plan.close()
