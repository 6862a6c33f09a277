"""Paged attention called again and again: split units, captured and concurrent calls and the device's reports, for both
types.  Bounds: tests/hybrid_reference.py."""
import itertools
import math

import pytest
import torch

import gated_deltanet_state_tail_b200 as gdn
import hybrid_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SENTINEL = 77.0


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Call:
    """A paged cache, queries and the arguments of one call over them."""

    def __init__(self, dtype, heads, kv, d, page, new, ctx, seed, width=None):
        self.new, self.ctx, self.dtype = new, ctx, dtype
        self.cache = ref.Paged(ctx, kv, d, page, dtype, seed, width=width)
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 + seed)
        self.q = torch.randn((sum(new), heads, d), generator=g, device="cuda").to(dtype)
        self.cu = [0] + list(itertools.accumulate(new))
        self.cu_t, self.ctx_t = _i32(self.cu), _i32(ctx)

    def attention(self):
        return gdn.PagedAttention(self.q.shape[1], self.cache.k.shape[2], self.q.shape[2], self.dtype, max_batch=len(self.ctx))

    def outputs(self):
        return torch.full_like(self.q, SENTINEL), torch.full(self.q.shape[:2], SENTINEL, device="cuda")

    def run(self, attn, o, lse=None, table=None, cu=None, ctx=None, **kw):
        attn.run(self.q, self.cache.k, self.cache.v, self.cache.table if table is None else table,
                 self.cu_t if cu is None else cu, self.ctx_t if ctx is None else ctx, o, lse, **kw)

    def check(self, o, lse, ctx=None):
        for (r0, r1), want, bound, want_lse, lse_bound in ref.attention(
                self.q, self.cache.k, self.cache.v, self.cache.table, self.cu, ctx or self.ctx, self.q.shape[2] ** -0.5, 0):
            assert bool(((o[r0:r1].double() - want).abs() <= bound).all()), (r0, r1)
            assert bool(((lse[r0:r1].double() - want_lse).abs() <= lse_bound).all()), (r0, r1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv,new", [(1, 1, 1), (8, 2, 1), (8, 1, 1), (8, 8, 1), (4, 2, 3), (8, 2, 2)])
def test_split_units_of_few_rows_over_and_over(dtype, d, heads, kv, new):
    """1 to 8 rows over a long context, cut over many CTAs: whoever merges has all of every part, so that each of many
    calls, from a workspace that holds NaN, gives the bits of the first."""
    call = Call(dtype, heads, kv, d, 16, [new], [9000 + 7 * heads + new], seed=d + heads + new)
    attn = call.attention()
    first, first_lse = call.outputs()
    call.run(attn, first, first_lse)
    attn.check()
    call.check(first, first_lse)
    outs = [call.outputs() for _ in range(40)]
    for o, lse in outs:
        attn.workspace.fill_(0xFF)   # a NaN in every word
        call.run(attn, o, lse)
    attn.check()
    for o, lse in outs:
        assert torch.equal(o, first) and torch.equal(lse, first_lse)


def _words(workspace):
    """The call number of the last launch, its arrival counts and its status word, in a workspace's header and behind it."""
    words = workspace[:512 + 8 * 296 * 8].view(torch.int64)
    return int(workspace[16:20].view(torch.int32)), words[512 // 8:], words[0:1]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_replays_after_a_launch_that_gave_up(dtype):
    """Arrival counts that a launch left short, under a status that says so (both written here): a replay merges nothing
    from parts that may not be in, keeps the status, and is right again once the workspace is zeroed."""
    call = Call(dtype, 8, 2, 128, 16, [1, 1], [9000, 30], seed=3)
    attn = call.attention()
    o, lse = call.outputs()
    call.run(attn, o, lse)
    attn.workspace.zero_()   # so that the words that this call does not use are told from those that it does
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(attn, o, lse)
    graph.replay()
    attn.check()
    good, good_lse = o.clone(), lse.clone()
    call.check(good, good_lse)
    number, counts, status = _words(attn.workspace)
    used = counts != 0
    assert bool(used.any()) and bool((counts[used] & 0xFFFFFFFF == 0).all())
    counts[used] += 1
    status.fill_((number << 32) | 2)
    o.fill_(SENTINEL)
    for _ in range(3):
        graph.replay()
        assert attn.status() == gdn.GDN_ERR_TIMEOUT
        assert bool((o[0] == SENTINEL).all()) and torch.equal(o[1], good[1])
    attn.workspace.zero_()
    graph.replay()
    assert attn.status() == gdn.GDN_OK and torch.equal(o, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("batch,rows", [(1, 1), (3, 40), (40, 700)])
def test_nothing_but_empty_sequences(dtype, batch, rows):
    """No sequence has a new token: every CTA ends without a piece of work, and the rows stay."""
    call = Call(dtype, 4, 2, 128, 16, [rows] + [0] * (batch - 1), [max(rows, 50)] * batch, seed=batch)
    attn = call.attention()
    o, lse = call.outputs()
    call.run(attn, o, lse, cu=_i32([0] * (batch + 1)))
    attn.check()
    assert bool((o == SENTINEL).all()) and bool((lse == SENTINEL).all())
    call.run(attn, o, lse)
    attn.check()
    call.check(o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx", [1, 128, 129, 640, 641, 1280, 1281, 3000])
@pytest.mark.parametrize("new", [1, 16, 40])
def test_every_copy_is_in_before_a_block_ends(d, ctx, new):
    """Pieces of one tile to more than the ring of copies holds, with and without tended value tiles, one after the other
    over the same rings: each copy's barrier completes as often as it is waited for."""
    call = Call(BF16, 8, 1, d, 16, [min(new, ctx)] * 3, [ctx] * 3, seed=ctx + new)
    attn = call.attention()
    o, lse = call.outputs()
    call.run(attn, o, lse)
    attn.check()
    call.check(o, lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_expanded_tensors_are_refused(dtype):
    """Through the public calls: nothing is launched, nothing written."""
    call = Call(dtype, 4, 2, 128, 16, [5], [30], seed=9)
    attn = call.attention()
    o, _ = call.outputs()
    call.q = call.q[:1].expand(5, 4, 128)
    with pytest.raises(ValueError):
        call.run(attn, o)
    x = torch.randn((5, 8, 128), device="cuda").to(dtype)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    pos, inv = torch.arange(5, device="cuda"), torch.ones(64, dtype=torch.float64, device="cuda")
    cache = dict(v=v, k_cache=call.cache.k, v_cache=call.cache.v, slots=pos)
    before = call.cache.k.clone()
    for kw in (dict(q=q[:1].expand_as(q), k=k, **cache), dict(q=q, k=k[:1].expand_as(k), **cache),
               dict(q=q, k=k, **dict(cache, v=v[:1].expand_as(v))),
               dict(q=q, k=k, **dict(cache, k_cache=x[0, 0].expand(3, 16, 2, 128), v_cache=x[0, 0].expand(3, 16, 2, 128)))):
        with pytest.raises(ValueError):
            gdn.qk_norm_rope(positions=pos, inv_freq=inv, **kw)
    torch.cuda.synchronize()
    assert bool((o == SENTINEL).all()) and torch.equal(call.cache.k.nan_to_num(), before.nan_to_num())


def _poke(call, b, key, head, column, value):
    page = call.cache.k.shape[1]
    call.cache.k[int(call.cache.table[b, key // page]), key % page, head, column] = value


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,heads,new,ctx", [(128, 2, 200, 200), (64, 2, 200, 200), (128, 8, 300, 300), (64, 8, 70, 150),
                                             (128, 16, 64, 4000), (128, 2, 3, 3000), (64, 8, 1, 130)])
def test_infinite_scores_make_a_row_nan(dtype, d, heads, new, ctx):
    """A key with an infinity scores +infinity with the rows whose query has its sign there: their softmax is NaN, at every
    position of a step and of the last one, in whole and in split units.  With the other sign the key has weight 0."""
    call = Call(dtype, heads, 2, d, 16, [new], [ctx], seed=d + new)
    call.q[..., 5] = torch.where(torch.arange(new, device="cuda")[:, None] % 3 == 0, -1.0, 1.0).to(dtype)
    attn = call.attention()
    good, good_lse = call.outputs()
    call.run(attn, good, good_lse)
    group, pos = heads // 2, torch.arange(ctx - new, ctx, device="cuda")
    keys = sorted({k for k in [*range(ctx - 70, ctx), *range(60, 70), 0, 1, 500, 1999] if 0 <= k < ctx})
    for key in keys:
        page, row = int(call.cache.table[0, key // 16]), key % 16
        was = call.cache.k[page, row, 1].clone()
        _poke(call, 0, key, 1, 5, math.inf)
        o, lse = call.outputs()
        call.run(attn, o, lse)
        call.cache.k[page, row, 1] = was
        nan = (pos >= key) & (torch.arange(new, device="cuda") % 3 != 0)
        assert bool(torch.isnan(o[nan, group:]).all()) and bool(torch.isnan(lse[nan, group:]).all()), key
        rest = ~nan & ((pos > 0) | (key > 0))   # a row with no other key has no softmax either
        assert bool(torch.isfinite(o[rest]).all()) and bool(torch.isfinite(lse[rest]).all()), key
        assert torch.equal(o[:, :group], good[:, :group]) and torch.equal(o[pos < key], good[pos < key])
    attn.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new,ctx", [(200, 200), (1, 300), (40, 40)])
def test_scores_beyond_fp32_do_not_vanish(dtype, new, ctx):
    """Finite products that overflow fp32 once scaled: NaN, as an infinite score, not a row of zeros."""
    call = Call(dtype, 4, 2, 128, 16, [new], [ctx], seed=17)
    call.q.fill_(2.0 ** 60)
    for key in range(ctx):
        _poke(call, 0, key, slice(None), slice(None), 1.0)
    attn = call.attention()
    o, lse = call.outputs()
    call.run(attn, o, lse, scale=2.0 ** 66)
    attn.check()
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,heads,new,ctx,window", [(128, 2, 200, 200, 0), (64, 8, 300, 300, 0), (128, 8, 40, 40, 0),
                                                    (128, 8, 300, 2000, 7), (64, 2, 3, 3000, 0), (128, 2, 1, 4000, 0),
                                                    (128, 4, 600, 3000, 0), (64, 8, 30, 20, 0)])
def test_rows_of_scores_of_minus_infinity_are_nan(dtype, d, heads, new, ctx, window):
    """-infinity for every key that a row sees is no softmax: o = NaN, lse = -infinity.  Beside other keys it is weight 0,
    bit for bit as a score far below theirs.  Rows without keys stay zero."""
    call = Call(dtype, heads, 2, d, 16, [new], [ctx], seed=d + new + 1)
    call.q[..., 5] = 1.0
    attn = call.attention()
    group, pos = heads // 2, torch.arange(ctx - new, ctx, device="cuda")
    keys = torch.arange(ctx, device="cuda")
    at = call.cache.table[0][keys // 16].long(), keys % 16
    was = call.cache.k.clone()
    for low, high in ((0, min(ctx, 10)), (ctx // 2, ctx // 2 + 9), (0, ctx // 2), (0, ctx - 1), (0, ctx)):
        got = {}
        hit = (keys >= low) & (keys < high)
        for value in (-math.inf, -4096.0):
            call.cache.k.copy_(was)
            call.cache.k[at[0][hit], at[1][hit], 1, 5] = value
            o, lse = call.outputs()
            call.run(attn, o, lse, window=window)
            got[value] = o, lse
        first = (pos - (window or ctx) + 1).clamp_min(0)
        gone = (pos >= 0) & (first >= low) & (pos < high)
        (o, lse), (far, far_lse) = got[-math.inf], got[-4096.0]
        assert bool(torch.isnan(o[gone, group:]).all()) and bool((lse[gone, group:] == -math.inf).all())
        assert torch.equal(o[~gone], far[~gone]) and torch.equal(lse[~gone], far_lse[~gone])
        assert torch.equal(o[:, :group], far[:, :group])
        assert bool((o[pos < 0] == 0).all()) and bool((lse[pos < 0] == -math.inf).all())
        assert bool(torch.isfinite(far).all())
    attn.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("how", ["argument", "current"])
def test_first_run_on_another_stream_than_the_workspace(dtype, how):
    """The workspace is made on one stream behind long work there, and first used on another: the call comes after its
    making, so that what the call reports is not wiped."""
    call = Call(dtype, 8, 2, 128, 16, [1, 20], [500, 90], seed=23)
    o, lse = call.outputs()
    call.run(call.attention(), o, lse)
    bad = call.cache.table.clone()
    bad[1, 1] = -1
    wrong, wrong_lse = call.outputs()
    again, again_lse = call.outputs()
    side = torch.cuda.Stream()
    a = torch.randn((8192, 8192), device="cuda", dtype=BF16)
    torch.cuda.synchronize()
    for _ in range(20):
        a @ a   # some 15 ms
    attn = call.attention()
    if how == "argument":
        call.run(attn, wrong, wrong_lse, table=bad, stream=side)
    else:
        with torch.cuda.stream(side):
            call.run(attn, wrong, wrong_lse, table=bad)
    torch.cuda.synchronize()
    assert attn.status() == gdn.GDN_ERR_MISMATCH
    call.run(attn, again, again_lse, stream=side)
    assert attn.status(side) == gdn.GDN_OK
    assert torch.equal(again, o) and torch.equal(again_lse, lse)


def test_workspace_outlives_its_calls_on_another_stream():
    """A PagedAttention that is dropped while its call waits on another stream: the memory is not handed out meanwhile."""
    call = Call(BF16, 8, 1, 128, 16, [1], [30000], seed=24)
    o, lse = call.outputs()
    call.run(call.attention(), o, lse)
    got, got_lse = call.outputs()
    side = torch.cuda.Stream()
    a = torch.randn((8192, 8192), device="cuda", dtype=BF16)
    attn = call.attention()
    size, at = attn.workspace.numel(), attn.workspace.data_ptr()
    call.run(attn, got, got_lse, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            a @ a
    call.run(attn, got, got_lse, stream=side)
    del attn
    taken = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != at for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(got, o) and torch.equal(got_lse, lse)


def test_reruns_of_fp32_give_the_same_bits():
    call = Call(F32, 8, 2, 128, 16, [1, 33, 260], [3000, 900, 2600], seed=41)
    attn = call.attention()
    first, first_lse = call.outputs()
    call.run(attn, first, first_lse)
    call.check(first, first_lse)
    for _ in range(10):
        attn.workspace.fill_(0xFF)
        o, lse = call.outputs()
        call.run(attn, o, lse)
        attn.check()
        assert torch.equal(o, first) and torch.equal(lse, first_lse)


def test_bad_descriptors_of_fp32_are_reported_and_skipped():
    """A page number outside the pool, a context past the table, offsets that decrease or leave the rows, for units of few
    rows and of many."""
    call = Call(F32, 4, 2, 128, 16, [20, 3, 1], [200, 90, 500], seed=61)
    attn = call.attention()
    good, good_lse = call.outputs()
    call.run(attn, good, good_lse)
    attn.check()
    for bad in (-1, call.cache.pages, 2 ** 31 - 1, -2 ** 31):
        for b, mine in ((0, slice(0, 20)), (1, slice(20, 23)), (2, slice(23, 24))):
            table = call.cache.table.clone()
            table[b, 2] = bad
            o, _ = call.outputs()
            call.run(attn, o, table=table)
            assert attn.status() == gdn.GDN_ERR_MISMATCH
            other = torch.ones(24, dtype=torch.bool, device="cuda")
            other[mine] = False
            assert torch.equal(o[other], good[other]) and bool(torch.isfinite(o[mine]).all())
    width = call.cache.table.shape[1] * 16
    for c in (width + 1, 2 ** 31 - 1, -1):
        o, _ = call.outputs()
        call.run(attn, o, ctx=_i32([200, c, 500]))
        assert attn.status() == gdn.GDN_ERR_MISMATCH
        assert bool((o[20:23] == SENTINEL).all()) and torch.equal(o[:20], good[:20]) and torch.equal(o[23:], good[23:])
    for offsets in ([0, 20, 23, 25], [0, 20, 23, 2 ** 31 - 1], [0, 20, 10, 24], [-1, 20, 23, 24]):
        o, _ = call.outputs()
        call.run(attn, o, cu=_i32(offsets))
        assert attn.status() == gdn.GDN_ERR_MISMATCH
    o, lse = call.outputs()
    call.run(attn, o, lse)
    assert attn.status() == gdn.GDN_OK and torch.equal(o, good) and torch.equal(lse, good_lse)


def test_captured_fp32_calls_follow_new_lengths():
    call = Call(F32, 8, 2, 128, 16, [1, 4, 20], [900, 60, 333], seed=71, width=80)
    ctx = _i32([5, 4, 20])
    attn, eager = call.attention(), call.attention()
    o, lse = call.outputs()
    call.run(attn, o, lse, ctx=ctx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(attn, o, lse, ctx=ctx)
    for lens in ([900, 60, 333], [17, 4, 100], [640, 33, 20], [900, 60, 333]):
        ctx.copy_(_i32(lens))
        for _ in range(3):
            o.fill_(SENTINEL)
            graph.replay()
        attn.check()
        want, want_lse = call.outputs()
        call.run(eager, want, want_lse, ctx=ctx)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
        call.check(o, lse, lens)


def test_two_fp32_calls_at_once():
    call = Call(F32, 8, 2, 128, 64, [1, 130, 2], [9000, 800, 5000], seed=81)
    want, want_lse = call.outputs()
    call.run(call.attention(), want, want_lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    attns = [call.attention() for _ in range(2)]
    outs = [call.outputs() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, a, (o, lse) in zip(streams, attns, outs):
            call.run(a, o, lse, stream=s)
    torch.cuda.synchronize()
    for s, a, (o, lse) in zip(streams, attns, outs):
        assert a.status(s) == gdn.GDN_OK and torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graphs_that_share_a_workspace_take_turns(dtype):
    """Two captured calls and an eager one of other shapes through one workspace, one after the other."""
    calls = [Call(dtype, 8, 2, 128, 16, new, ctx, seed=51 + n) for n, (new, ctx) in
             enumerate([([1, 1], [9000, 70]), ([2, 5], [400, 3000]), ([300], [2500])])]
    attn = calls[0].attention()
    outs, want = [c.outputs() for c in calls], [c.outputs() for c in calls]
    graphs = []
    for c, (o, lse), w in zip(calls, outs, want):
        c.run(c.attention(), *w)
        c.run(attn, o, lse)
        if c is not calls[2]:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                c.run(attn, o, lse)
    for turn in range(6):
        for n in ((0, 1, 2), (2, 1, 0), (1, 1, 0))[turn % 3]:
            outs[n][0].fill_(SENTINEL)
            graphs[n].replay() if n < 2 else calls[2].run(attn, *outs[2])
            assert attn.status() == gdn.GDN_OK
            assert torch.equal(outs[n][0], want[n][0]) and torch.equal(outs[n][1], want[n][1])


def test_misaligned_index_arrays_are_refused_by_name():
    call = Call(BF16, 4, 2, 128, 16, [1, 1, 1], [30, 40, 50], seed=9)
    attn = call.attention()
    o, _ = call.outputs()
    longer = _i32([0] + call.ctx)
    with pytest.raises(gdn.GdnError, match="context_len must start"):
        call.run(attn, o, ctx=longer[1:])
    call.run(attn, o, ctx=longer[1:].clone())
    attn.check()
    x = torch.randn((3, 8, 128), device="cuda").to(BF16)
    pos, inv = torch.arange(4, device="cuda"), torch.ones(64, dtype=torch.float64, device="cuda")
    with pytest.raises(gdn.GdnError, match="positions, slots must start"):
        gdn.qk_norm_rope(x[:, :4], x[:, 4:6], pos[1:], inv, v=x[:, 6:], k_cache=call.cache.k, v_cache=call.cache.v, slots=pos[1:])


def test_a_unit_of_more_than_a_second():
    """One token over 250 million keys (few pages, again and again), a key head per CTA: a unit takes longer than the
    second that a wait may take for short contexts.  Values are not compared: fp32 sums of as many terms are not exact."""
    heads, d, page, pages, times = 148, 64, 256, 4, 250_000
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k, v = (torch.randn((pages, page, heads, d), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((1, heads, d), generator=g, device="cuda").to(BF16)
    attn = gdn.PagedAttention(heads, heads, d, BF16, max_batch=1)
    got = []
    for n in (1, times):
        table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n)[None]
        o, lse = torch.full_like(q, SENTINEL), torch.full((1, heads), SENTINEL, device="cuda")
        attn.run(q, k, v, table, _i32([0, 1]), _i32([n * pages * page]), o, lse)
        assert attn.status() == gdn.GDN_OK
        got.append((o.float(), lse))
    assert bool(torch.isfinite(got[1][0]).all())
    # a rounded sum of positive terms never shrinks: at least one repeat's log-sum, up to its own 1024 roundings
    assert bool((got[1][1] >= got[0][1] - 1e-3).all())
