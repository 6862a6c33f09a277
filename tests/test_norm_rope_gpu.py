"""gdn_qk_norm_rope against a plain 64-bit implementation.  Bounds: tests/hybrid_reference.py."""
import math

import pytest
import torch

import gated_deltanet_state_tail_b200 as gdn
import hybrid_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _inputs(dtype, rows, heads, kv, d, rot, far, seed, fused=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn((rows, heads + 2 * kv, d), generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(max(0, far - 5000), far + 1, (rows,), generator=g, device="cuda")
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot) if rot else None
    qw = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    kw = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    return q, k, v, pos, inv, qw, kw


def _close(got, want_bound, what):
    want, bound = want_bound
    off = (got.double() - want).abs() / (bound + 1e-30)
    assert bool((off <= 1).all()), f"{what}: {float(off.nan_to_num(nan=math.inf).max())} of the bound"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,kv", [(1, 16, 4), (7, 5, 1), (297, 6, 2), (1301, 3, 3)])
def test_norm_and_rotation(dtype, d, rot, interleaved, rows, heads, kv):
    q, k, v, pos, inv, qw, kw = _inputs(dtype, rows, heads, kv, d, rot, 40000, rows + d + rot)
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw, eps=1e-6, interleaved=interleaved)
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-6, interleaved), "q")
    _close(ko, ref.norm_rope(k, pos, inv, kw, 1e-6, interleaved), "k")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_rows(dtype, d, interleaved):
    """Enough rows for the widest row blocks, the last block not full, and keys and values appended."""
    rows, heads, kv, page = 4741, 5, 3, 16
    q, k, v, pos, inv, qw, kw = _inputs(dtype, rows, heads, kv, d, 32, 40000, 8)
    pages = -(-rows // page)
    kc = torch.full((pages, page, kv, d), 7.0, dtype=dtype, device="cuda")
    vc = torch.full_like(kc, 7.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:rows]
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw, interleaved=interleaved, v=v, k_cache=kc, v_cache=vc, slots=slots,
                              k_out=torch.empty((rows, kv, d), dtype=dtype, device="cuda"))
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-6, interleaved), "q")
    _close(ko, ref.norm_rope(k, pos, inv, kw, 1e-6, interleaved), "k")
    assert torch.equal(kc.view(-1, kv, d)[slots], ko) and torch.equal(vc.view(-1, kv, d)[slots], v)
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert bool((kc.view(-1, kv, d)[rest] == 7).all()) and bool((vc.view(-1, kv, d)[rest] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("far", [0, 1, 131072, 10 ** 6, 2 ** 31, 2 ** 40])
def test_far_positions(dtype, far):
    q, k, v, pos, inv, qw, kw = _inputs(dtype, 33, 4, 2, 128, 128, far, 5)
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw)
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-6, False), "q")
    _close(ko, ref.norm_rope(k, pos, inv, kw, 1e-6, False), "k")


@pytest.mark.parametrize("freq", [0.0, -0.37, 1.0, 6.5, 40.0])
def test_any_frequency(freq):
    """Negative frequencies and ones of more than a turn per position."""
    q, k, v, pos, inv, qw, kw = _inputs(F32, 21, 2, 2, 64, 32, 3000, 6)
    inv = torch.full_like(inv, freq)
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw)
    # the frequency itself is rounded to 2^-52 of it on the way to turns
    want, bound = ref.norm_rope(q, pos, inv, qw, 1e-6, False)
    _close(qo, (want, bound + 3000 * abs(freq) * 2.0 ** -50 * 10), "q")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which", ["none", "q", "k"])
def test_without_weights(dtype, which):
    q, k, v, pos, inv, qw, kw = _inputs(dtype, 40, 4, 2, 128, 64, 900, 7)
    qw, kw = (qw if which == "q" else None), (kw if which == "k" else None)
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw)
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-6, False), "q")
    _close(ko, ref.norm_rope(k, pos, inv, kw, 1e-6, False), "k")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_small_and_large_heads(dtype):
    """Heads of zeros, tiny and huge values: eps decides at zero, the sum of squares stays finite in fp32."""
    q, k, v, pos, inv, qw, kw = _inputs(dtype, 12, 4, 2, 128, 128, 900, 8, fused=False)
    q[0] = 0
    q[1] *= 1e-12
    q[2] *= 1e15
    qo, _ = gdn.qk_norm_rope(q, k, pos, inv, qw, kw, eps=1e-5)
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-5, False), "q")
    assert bool((qo[0] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_stays_in_its_head(dtype):
    q, k, v, pos, inv, qw, kw = _inputs(dtype, 9, 4, 2, 128, 64, 900, 9, fused=False)
    q[3, 1, 5] = math.nan
    k[4, 0, 100] = math.inf
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw)
    bad = ~torch.isfinite(qo).all(-1)
    assert bad.nonzero().tolist() == [[3, 1]]
    assert (~torch.isfinite(ko).all(-1)).nonzero().tolist() == [[4, 0]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(dtype, interleaved):
    q, k, v, pos, inv, qw, kw = _inputs(dtype, 500, 6, 2, 128, 96, 900, 10, fused=False)
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw, interleaved=interleaved)
    q2, k2 = q.clone(), k.clone()
    gdn.qk_norm_rope(q2, k2, pos, inv, qw, kw, interleaved=interleaved, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["packed", "heads first", "pairs"])
@pytest.mark.parametrize("rows", [1, 70, 900])
def test_append(dtype, layout, rows):
    """Keys and values land in their slots, rows with a slot outside the pool nowhere, and nothing else changes."""
    heads, kv, d, page = 4, 2, 128, 24
    q, k, v, pos, inv, qw, kw = _inputs(dtype, rows, heads, kv, d, 64, 5000, 11)
    cache = ref.Paged([rows + 100], kv, d, page, dtype, 12, layout)
    slots = torch.randperm(cache.pages * page, device="cuda")[:rows]
    if rows > 4:
        slots[0], slots[1], slots[2], slots[3] = -1, cache.pages * page, 2 ** 62, -2 ** 62
    before_k, before_v = cache.k.clone(), cache.v.clone()
    k_out = torch.zeros((rows, kv, d), dtype=dtype, device="cuda")
    qo, ko = gdn.qk_norm_rope(q, k, pos, inv, qw, kw, v=v, k_cache=cache.k, v_cache=cache.v, slots=slots, k_out=k_out)
    assert ko is k_out
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-6, False), "q")
    _close(ko, ref.norm_rope(k, pos, inv, kw, 1e-6, False), "k")
    ok = (slots >= 0) & (slots < cache.pages * page)
    at = (slots[ok] // page, slots[ok] % page)
    assert torch.equal(cache.k[at], k_out[ok]) and torch.equal(cache.v[at], v[ok])
    before_k[at], before_v[at] = cache.k[at], cache.v[at]

    def same(x, y):
        return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))

    assert same(before_k, cache.k) and same(before_v, cache.v)


def test_slots_beyond_32_bits():
    page, kv, d = 64, 8, 128
    pages = 2 ** 32 // (page * kv * d) + 5
    free, _ = torch.cuda.mem_get_info()
    if free < 2 * pages * page * kv * d * 2 + 2 ** 31:
        pytest.skip("not enough free memory")
    kc = torch.empty((pages, page, kv, d), dtype=BF16, device="cuda")
    vc = torch.empty((pages, page, kv, d), dtype=BF16, device="cuda")
    q, k, v, pos, inv, qw, kw = _inputs(BF16, 50, 8, kv, d, 128, 5000, 13)
    slots = pages * page - 1 - torch.arange(50, device="cuda")
    k_out = torch.empty((50, kv, d), dtype=BF16, device="cuda")
    gdn.qk_norm_rope(q, k, pos, inv, qw, kw, v=v, k_cache=kc, v_cache=vc, slots=slots, k_out=k_out)
    assert torch.equal(kc[slots // page, slots % page], k_out) and torch.equal(vc[slots // page, slots % page], v)


def test_captured_call_follows_new_positions():
    q, k, v, pos, inv, qw, kw = _inputs(BF16, 8, 4, 2, 128, 128, 100, 14)
    cache = ref.Paged([64], 2, 128, 16, BF16, 15)
    slots = torch.arange(8, device="cuda")
    qo = torch.empty((8, 4, 128), dtype=BF16, device="cuda")
    args = dict(v=v, k_cache=cache.k, v_cache=cache.v, slots=slots, q_out=qo)
    gdn.qk_norm_rope(q, k, pos, inv, qw, kw, **args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.qk_norm_rope(q, k, pos, inv, qw, kw, **args)
    pos += 777
    slots += 20
    graph.replay()
    _close(qo, ref.norm_rope(q, pos, inv, qw, 1e-6, False), "q")
    _close(cache.k.view(-1, 2, 128)[slots], ref.norm_rope(k, pos, inv, kw, 1e-6, False), "k")
