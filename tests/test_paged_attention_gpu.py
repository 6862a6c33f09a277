"""gdn_paged_attention against a plain 64-bit implementation: lengths from none to long, groups, pages, windows,
strides, and what the device checks refuse.  Bounds: tests/hybrid_reference.py."""
import itertools
import math

import pytest
import torch

import gated_deltanet_state_tail_b200 as gdn
import hybrid_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SENTINEL = 77.0


def _queries(new, heads, d, dtype, seed, scale=1.0, strided=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 + seed)
    rows = sum(new)
    if strided:   # the first heads of a wider projection
        wide = torch.randn((rows, heads + 3, d), generator=g, device="cuda") * scale
        return wide.to(dtype)[:, :heads]
    return (torch.randn((rows, heads, d), generator=g, device="cuda") * scale).to(dtype)


def _cu(new):
    return [0] + list(itertools.accumulate(new))


def _run(q, cache, cu, ctx, window=0, scale=None, attn=None, extra=3):
    """o and lse of q's rows, with `extra` rows behind the last sequence that must stay as they were."""
    rows, heads, d = q.shape
    if extra:
        q = torch.cat([q, torch.full((extra, heads, d), math.nan, dtype=q.dtype, device="cuda")])
    o = torch.full((rows + extra, heads, d), SENTINEL, dtype=q.dtype, device="cuda")
    lse = torch.full((rows + extra, heads), SENTINEL, device="cuda")
    attn = attn or gdn.PagedAttention(heads, cache.k.shape[2], d, q.dtype, max_batch=len(ctx))
    attn.run(q, cache.k, cache.v, cache.table, torch.tensor(cu, dtype=torch.int32, device="cuda"),
             torch.tensor(ctx, dtype=torch.int32, device="cuda"), o, lse, scale=scale, window=window)
    assert attn.status() == gdn.GDN_OK
    assert bool((o[rows:] == SENTINEL).all()) and bool((lse[rows:] == SENTINEL).all())
    return o[:rows], lse[:rows]


def _check(q, cache, cu, ctx, o, lse, window=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    worst = 0.0
    for (r0, r1), want, bound, want_lse, lse_bound in ref.attention(q, cache.k, cache.v, cache.table, cu, ctx, scale, window):
        off = (o[r0:r1].double() - want).abs() / bound
        assert bool((off <= 1).all()), f"rows {r0}:{r1}: {float(off.nan_to_num(nan=math.inf).max())} of the bound"
        worst = max(worst, float(off.max()))
        got = lse[r0:r1].double()
        none = torch.isinf(want_lse)
        assert torch.equal(torch.isinf(got) & (got < 0), none)
        off = torch.where(none, 0.0, (got - want_lse).abs() / lse_bound)
        assert bool((off <= 1).all()), f"lse of rows {r0}:{r1}: {float(off.nan_to_num(nan=math.inf).max())} of the bound"
    return worst


def _case(dtype, heads, kv, d, page, new, ctx, window=0, scale=None, seed=0, layout="packed", q_scale=1.0, k_scale=1.0,
          strided=False):
    cache = ref.Paged(ctx, kv, d, page, dtype, seed, layout, k_scale)
    q = _queries(new, heads, d, dtype, seed, q_scale, strided)
    cu = _cu(new)
    o, lse = _run(q, cache, cu, ctx, window, scale, extra=0 if strided else 3)
    _check(q, cache, cu, ctx, o, lse, window, scale)
    return q, cache, cu, o, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv,page", [(8, 8, 16), (16, 2, 64), (6, 2, 48), (7, 1, 8)])
def test_single_tokens(dtype, d, heads, kv, page):
    ctx = [1, 2, 15, 16, 17, 127, 128, 129, 0, 255, 257, 1000, 4097]
    _case(dtype, heads, kv, d, page, [1] * len(ctx), ctx, seed=d + page)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv,page", [(4, 4, 32), (8, 2, 16), (5, 1, 256), (12, 4, 24)])
def test_chunks(dtype, d, heads, kv, page):
    new = [1, 5, 16, 0, 17, 33, 64, 100, 129, 300, 0]
    ctx = [700, 5, 129, 40, 256, 1000, 64, 101, 130, 2000, 0]
    _case(dtype, heads, kv, d, page, new, ctx, seed=3 * d + page)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [1, 2, 7, 64, 128, 200, 5000])
def test_windows(dtype, window):
    new = [1, 40, 130, 260, 1]
    ctx = [900, 333, 130, 1500, 3]
    _case(dtype, 6, 2, 64, 16, new, ctx, window=window, seed=window)
    _case(dtype, 2, 2, 128, 64, new, ctx, window=window, seed=window + 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pages_before_the_window_are_not_read(dtype):
    """Page numbers of pages that no row's window reaches are garbage; rows before the window hold NaN."""
    page, window, ctx, new = 16, 40, [500, 333, 1111], [1, 20, 150]
    cache = ref.Paged(ctx, 2, 128, page, dtype, 5)
    q, cu = _queries(new, 4, 128, dtype, 5), _cu(new)
    want = list(ref.attention(q, cache.k, cache.v, cache.table, cu, ctx, 128 ** -0.5, window))
    for b, (n, c) in enumerate(zip(new, ctx)):
        lo = max(0, c - n - window + 1)
        i = torch.arange(lo, device="cuda")
        pages = cache.table[b][i // page].long()
        cache.k[pages, i % page] = math.nan
        cache.v[pages, i % page] = math.inf
        cache.table[b, :lo // page] = -5
    o, lse = _run(q, cache, cu, ctx, window)
    for (r0, r1), w, bound, _, _ in want:
        assert bool(((o[r0:r1].double() - w).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_without_keys(dtype):
    """More new tokens than context: the rows before position 0 see nothing."""
    new, ctx = [10, 200, 3, 150], [4, 0, 3, 149]
    q, cache, cu, o, lse = _case(dtype, 4, 2, 128, 16, new, ctx)
    assert bool((o[:6] == 0).all()) and bool(torch.isinf(lse[:6]).all())
    assert bool((o[10:210] == 0).all()) and bool(torch.isinf(lse[10:210]).all())
    assert bool(torch.isfinite(lse[6:10]).all())


@pytest.mark.parametrize("dtype,heads,kv", [(BF16, 64, 1), (F32, 64, 1), (BF16, 33, 1), (BF16, 22, 2), (F32, 48, 2)])
def test_large_groups(dtype, heads, kv):
    _case(dtype, heads, kv, 64, 16, [1, 7, 40], [300, 77, 200], seed=heads)
    _case(dtype, heads, kv, 128, 32, [3, 1], [140, 1025], seed=heads + 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["heads first", "pairs"])
def test_cache_layouts_and_strided_queries(dtype, layout):
    new, ctx = [1, 50, 9], [400, 333, 9]
    _case(dtype, 8, 4, 128, 16, new, ctx, layout=layout, strided=True, seed=8)
    _case(dtype, 8, 4, 64, 40, new, ctx, layout=layout, strided=True, window=100, seed=9)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_scale", [0.01, 4.0, 30.0])
def test_score_ranges(dtype, q_scale):
    """Flat, peaked and one-hot softmax rows; the maximum keeps growing along the keys."""
    new, ctx = [1, 130], [1500, 700]
    cache = ref.Paged(ctx, 2, 128, 64, dtype, 11)
    for b, c in enumerate(ctx):   # later keys are larger
        i = torch.arange(c, device="cuda")
        rows = cache.table[b][i // 64].long(), i % 64
        cache.k[rows] = (cache.k[rows].float() * (0.05 + 2 * i / c)[:, None, None]).to(dtype)
    q, cu = _queries(new, 4, 128, dtype, 12, q_scale), _cu(new)
    o, lse = _run(q, cache, cu, ctx)
    _check(q, cache, cu, ctx, o, lse)


@pytest.mark.parametrize("scale", [1.0, 0.02, 1e-8])
def test_scale(scale):
    _case(BF16, 4, 2, 64, 16, [1, 40], [200, 300], scale=scale, q_scale=0.2, seed=21)
    _case(F32, 4, 2, 64, 16, [1, 40], [200, 300], scale=scale, q_scale=0.2, seed=22)


@pytest.mark.parametrize("dtype,new,ctx", [
    (BF16, [1], [40001]), (F32, [1], [20011]), (BF16, [3, 1, 2], [9000, 30000, 129]), (BF16, [520], [8712]),
    (F32, [65], [5000]), (BF16, [1500], [1500]), (BF16, [1] * 300, list(range(1, 301))),
])
def test_long_and_many(dtype, new, ctx):
    _case(dtype, 8, 2, 128, 64, new, ctx, seed=len(ctx))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_sequences_than_one_scan_block(dtype):
    """The schedule's scan over the sequences takes several rounds."""
    batch = 2500
    new = [i % 3 for i in range(batch)]
    ctx = [(7 * i) % 60 + 2 for i in range(batch)]
    cache = ref.Paged(ctx, 1, 64, 8, dtype, 31)
    q, cu = _queries(new, 2, 64, dtype, 31), _cu(new)
    o, lse = _run(q, cache, cu, ctx)
    _check(q, cache, cu, ctx, o, lse)


def test_reruns_give_the_same_bits():
    new, ctx = [1, 33, 260], [3000, 900, 2600]
    cache = ref.Paged(ctx, 2, 128, 16, BF16, 41)
    q, cu = _queries(new, 8, 128, BF16, 41), _cu(new)
    attn = gdn.PagedAttention(8, 2, 128, BF16, max_batch=3)
    first = _run(q, cache, cu, ctx, attn=attn)
    attn.workspace.fill_(0xFF)   # needs no initialisation
    again = _run(q, cache, cu, ctx, attn=attn)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_without_lse_and_one_shot():
    new, ctx = [1, 33], [300, 90]
    cache = ref.Paged(ctx, 2, 128, 16, BF16, 42)
    q, cu = _queries(new, 8, 128, BF16, 42), _cu(new)
    o, lse = _run(q, cache, cu, ctx)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (q, cache.k, cache.v, cache.table, torch.tensor(cu, **i32), torch.tensor(ctx, **i32))
    assert torch.equal(gdn.paged_attention(*args), o)
    o2, lse2 = gdn.paged_attention(*args, with_lse=True)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_beyond_32_bits(dtype):
    """A pool of more than 2^32 elements: pages at its far end."""
    page, kv, d = 64, 8, 128
    per_page = 2 * page * kv * d
    pages = 2 ** 32 // per_page + 40
    free, _ = torch.cuda.mem_get_info()
    need = pages * per_page * (2 if dtype == BF16 else 4)
    if free < need + 2 ** 31:
        pytest.skip("not enough free memory")
    pool = torch.empty((pages, 2, page, kv, d), dtype=dtype, device="cuda")
    k, v = pool[:, 0], pool[:, 1]
    ctx, new = [600, 70], [1, 20]
    cache = ref.Paged(ctx, kv, d, page, dtype, 51)
    far = pages - 1 - torch.arange(cache.pages, device="cuda")
    k[far], v[far] = cache.k, cache.v
    cache.k, cache.v = k, v
    cache.table = torch.where(cache.table < cache.pages, pages - 1 - cache.table, cache.table)
    q, cu = _queries(new, 16, d, dtype, 51), _cu(new)
    o, lse = _run(q, cache, cu, ctx)
    _check(q, cache, cu, ctx, o, lse)


def test_bad_descriptors_are_reported_and_skipped():
    """A page number outside the pool, a context past the table, offsets that decrease or leave the rows: the status
    says so, rows of sequences that cannot be placed stay, and the other sequences are right."""
    new, ctx = [20, 3, 1], [200, 90, 500]
    cache = ref.Paged(ctx, 2, 128, 16, BF16, 61)
    q, cu = _queries(new, 4, 128, BF16, 61), _cu(new)
    good, _ = _run(q, cache, cu, ctx)
    attn = gdn.PagedAttention(4, 2, 128, BF16, max_batch=3)
    i32 = dict(dtype=torch.int32, device="cuda")

    def run(table=cache.table, cu=cu, ctx=ctx):
        o = torch.full(q.shape, SENTINEL, dtype=BF16, device="cuda")
        attn.run(q, cache.k, cache.v, table, torch.tensor(cu, **i32), torch.tensor(ctx, **i32), o)
        return o, attn.status()

    for bad in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):
        table = cache.table.clone()
        table[1, 2] = bad
        o, status = run(table=table)
        assert status == gdn.GDN_ERR_MISMATCH
        assert torch.equal(o[:20], good[:20]) and torch.equal(o[23:], good[23:])
        assert bool(torch.isfinite(o[20:23]).all())
    width = cache.table.shape[1] * 16
    for c in (width + 1, 2 ** 31 - 1, -1):
        o, status = run(ctx=[200, c, 500])
        assert status == gdn.GDN_ERR_MISMATCH
        assert bool((o[20:23] == SENTINEL).all()) and torch.equal(o[:20], good[:20]) and torch.equal(o[23:], good[23:])
    for offsets in ([0, 20, 23, 25], [0, 20, 23, 2 ** 31 - 1], [0, 20, 10, 24], [-1, 20, 23, 24]):
        o, status = run(cu=offsets)
        assert status == gdn.GDN_ERR_MISMATCH
    o, status = run()
    assert status == gdn.GDN_OK and torch.equal(o, good)


def test_captured_call_follows_new_lengths():
    """A captured call replayed with other lengths, pages and values gives what an eager call gives."""
    ctx, new = [900, 60, 333], [1, 4, 20]
    cache = ref.Paged(ctx, 2, 128, 16, BF16, 71, width=80)
    q, cu = _queries(new, 8, 128, BF16, 71), _cu(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_t, ctx_t = torch.tensor(cu, **i32), torch.tensor([5, 4, 20], **i32)
    o = torch.zeros_like(q)
    attn = gdn.PagedAttention(8, 2, 128, BF16, max_batch=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attn.run(q, cache.k, cache.v, cache.table, cu_t, ctx_t, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.run(q, cache.k, cache.v, cache.table, cu_t, ctx_t, o)
    for lens in ([900, 60, 333], [17, 4, 100], [640, 33, 20]):
        ctx_t.copy_(torch.tensor(lens, **i32))
        graph.replay()
        torch.cuda.synchronize()
        eager, _ = _run(q, cache, cu, lens, extra=0)
        assert torch.equal(o, eager)


def test_two_calls_at_once():
    """Two streams with a workspace each, against the same calls one after the other."""
    ctx, new = [9000, 800], [1, 130]
    cache = ref.Paged(ctx, 2, 128, 64, BF16, 81)
    q, cu = _queries(new, 8, 128, BF16, 81), _cu(new)
    want, _ = _run(q, cache, cu, ctx)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_t, ctx_t = torch.tensor(cu, **i32), torch.tensor(ctx, **i32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    attns = [gdn.PagedAttention(8, 2, 128, BF16, max_batch=2) for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, a, o in zip(streams, attns, outs):
            a.run(q, cache.k, cache.v, cache.table, cu_t, ctx_t, o, stream=s)
    torch.cuda.synchronize()
    for a, o in zip(attns, outs):
        assert a.status() == gdn.GDN_OK and torch.equal(o, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_chunks_follow_new_lengths(dtype):
    """As above with chunks of many rows: units that the schedule splits over CTAs at one length and not at another."""
    new, ctx = [200, 70], [2600, 70]
    cache = ref.Paged(ctx, 2, 128, 32, dtype, 72, width=90)
    q, cu = _queries(new, 8, 128, dtype, 72), _cu(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_t, ctx_t = torch.tensor(cu, **i32), torch.tensor(ctx, **i32)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    attn = gdn.PagedAttention(8, 2, 128, dtype, max_batch=2)
    attn.run(q, cache.k, cache.v, cache.table, cu_t, ctx_t, o, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.run(q, cache.k, cache.v, cache.table, cu_t, ctx_t, o, lse)
    for lens in ([2600, 70], [200, 70], [1031, 70], [2600, 70]):
        ctx_t.copy_(torch.tensor(lens, **i32))
        for _ in range(2):
            o.fill_(SENTINEL)
            graph.replay()
        torch.cuda.synchronize()
        eager, eager_lse = _run(q, cache, cu, lens, extra=0)
        assert torch.equal(o, eager) and torch.equal(lse, eager_lse)
        _check(q, cache, cu, lens, o, lse)


def test_one_workspace_for_calls_of_other_sizes():
    """Batches, head dims and dtypes in turn through one workspace of arbitrary bytes, small numbers among them."""
    size = max(gdn.gdn_paged_attention_workspace_bytes(t, d, 400) for t in ("bf16", "f32") for d in (64, 128))
    workspace = torch.arange(size // 4, dtype=torch.int32, device="cuda") % 512
    cases = [(BF16, 128, [1, 1, 1], [3000, 90, 2049]), (F32, 64, [20] * 5, [700] * 5), (BF16, 64, [150] * 9, [900] * 9),
             (BF16, 128, [1] * 400, [130] * 400), (F32, 128, [1, 2], [1500, 4000]), (BF16, 128, [300], [5000])]
    for turn in range(3):
        for n, (dtype, d, new, ctx) in enumerate(cases):
            cache = ref.Paged(ctx, 2, d, 16, dtype, 90 + n)
            q, cu = _queries(new, 8, d, dtype, 90 + n), _cu(new)
            i32 = dict(dtype=torch.int32, device="cuda")
            args = (torch.tensor(cu, **i32), torch.tensor(ctx, **i32))
            o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
            gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, *args, o, lse, workspace)
            assert gdn.gdn_workspace_status(workspace) == gdn.GDN_OK
            if turn == 0:
                _check(q, cache, cu, ctx, o, lse)
            want, want_lse = _run(q, cache, cu, ctx, extra=0)
            assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_queries_and_keys_stay_in_their_rows(dtype, bad):
    """A NaN or infinity in one query changes no other row; one in a key changes no row that does not see it."""
    new, ctx = [70, 1, 40], [300, 500, 40]
    cache = ref.Paged(ctx, 2, 128, 16, dtype, 95)
    q, cu = _queries(new, 4, 128, dtype, 95), _cu(new)
    good, good_lse = _run(q, cache, cu, ctx)
    x = q.clone()
    x[33, 1, 7] = bad
    o, lse = _run(x, cache, cu, ctx)
    changed = (o != good).any(-1) | (lse != good_lse)
    assert not bool(torch.isfinite(o[33, 1]).all())
    changed[33, 1] = False
    assert not bool(changed.any())
    # key 20 of the third request (rows 71 .. 110 are its positions 0 .. 39), head 1 of two
    page, row = int(cache.table[2, 20 // 16]), 20 % 16
    cache.k[page, row, 1, 3] = bad
    o, lse = _run(q, cache, cu, ctx)
    same = (o == good).all(-1) & (lse == good_lse)
    assert bool(same[:71 + 20].all()) and bool(same[:, :2].all())
    if math.isnan(bad):
        assert bool(torch.isnan(o[71 + 20:, 2:]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,heads,window", [(128, 4, 0), (64, 2, 0), (128, 16, 0), (64, 12, 90), (128, 2, 33)])
def test_bad_values_reach_only_rows_that_see_them(dtype, bad, d, heads, window):
    """A value that is not finite, in one column of one key: rows that see the key have it in that column, nothing else
    of any row changes by a bit."""
    new, ctx = [70, 1, 300, 6], [300, 500, 2000, 6]
    cache = ref.Paged(ctx, 2, d, 16, dtype, 96)
    q, cu = _queries(new, heads, d, dtype, 96), _cu(new)
    good, good_lse = _run(q, cache, cu, ctx, window)
    group = heads // 2
    for b, pos in ((0, 260), (0, 299), (2, 1701), (2, 1850), (2, 1999), (3, 0), (3, 5), (1, 499), (2, 1650)):
        at = (int(cache.table[b, pos // 16]), pos % 16, 1, 7)
        was = cache.v[at].clone()
        cache.v[at] = bad
        o, lse = _run(q, cache, cu, ctx, window)
        cache.v[at] = was
        first = ctx[b] - new[b]
        rows = torch.arange(cu[b], cu[b + 1], device="cuda")
        row_pos = rows - cu[b] + first
        sees = rows[(row_pos >= pos) & ((row_pos - pos < window) | (window == 0))]
        want = good.clone()
        want[sees, group:, 7] = bad
        assert torch.equal(o.nan_to_num(nan=1e9), want.nan_to_num(nan=1e9)), (b, pos)
        assert torch.equal(lse, good_lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_padded_chunks(dtype):
    """A padded batch: every request has 64 rows, its real tokens first; what the padding holds reaches no real row."""
    real, ctx_real = [64, 10, 1, 33], [500, 10, 77, 1033]
    new = [64] * 4
    ctx = [c - r + 64 for c, r in zip(ctx_real, real)]      # the padding's rows are in the cache too
    cache = ref.Paged(ctx, 2, 128, 16, dtype, 97)
    q, cu = _queries(new, 8, 128, dtype, 97), _cu(new)
    want = {}
    for b, (r, c) in enumerate(zip(real, ctx_real)):
        for (r0, r1), o, bound, _, _ in ref.attention(q[cu[b]:cu[b] + r], cache.k, cache.v, cache.table[b:b + 1], [0, r], [c],
                                                      128 ** -0.5, 0):
            want[b] = (o, bound)
        at = torch.arange(c, ctx[b], device="cuda")
        rows = cache.table[b][at // 16].long(), at % 16
        cache.k[rows], cache.v[rows] = math.nan, math.inf
        q[cu[b] + r:cu[b + 1]] = math.nan
    o, _ = _run(q, cache, cu, ctx)
    for b, r in enumerate(real):
        w, bound = want[b]
        assert bool(((o[cu[b]:cu[b] + r].double() - w).abs() <= bound).all()), b


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 300, 1000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_windows_beyond_every_context(dtype, window):
    """A window that no context reaches changes nothing, for rows without keys beside rows with some too."""
    new, ctx = [300, 1, 40], [120, 999, 700]
    cache = ref.Paged(ctx, 2, 64, 16, dtype, 91)
    q, cu = _queries(new, 6, 64, dtype, 91), _cu(new)
    o, lse = _run(q, cache, cu, ctx, window)
    _check(q, cache, cu, ctx, o, lse)
    all_o, all_lse = _run(q, cache, cu, ctx)
    assert torch.equal(o, all_o) and torch.equal(lse, all_lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_contexts_beyond_the_largest_are_reported(dtype):
    cache = ref.Paged([50, 50], 1, 64, 8, dtype, 92)
    q = _queries([1, 1], 1, 64, dtype, 92)
    good, _ = _run(q, cache, [0, 1, 2], [50, 50])
    table = torch.zeros((2, 2 ** 27 + 1), dtype=torch.int32, device="cuda")   # room for 2^30 + 8 keys a row
    table[:, :cache.table.shape[1]] = cache.table
    attn = gdn.PagedAttention(1, 1, 64, dtype, max_batch=2)
    i32 = dict(dtype=torch.int32, device="cuda")
    o = torch.full(q.shape, SENTINEL, dtype=dtype, device="cuda")
    attn.run(q, cache.k, cache.v, table, torch.tensor([0, 1, 2], **i32), torch.tensor([50, 2 ** 30 + 1], **i32), o)
    assert attn.status() == gdn.GDN_ERR_MISMATCH
    assert torch.equal(o[:1], good[:1]) and bool((o[1:] == SENTINEL).all())
