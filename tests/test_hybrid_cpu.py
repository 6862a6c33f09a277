"""Refusals of the full-attention operators: every argument check answers before any device work."""
import ctypes

import pytest
import torch

import gated_deltanet_state_tail_b200 as gdn

OK, INVALID, UNSUPPORTED = gdn.GDN_OK, gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED
PTR = 4096   # an aligned address that a refused call never reads


def _cache(**kw):
    c = gdn.gdn_paged_kv()
    c.num_pages, c.page_size, c.num_kv_heads, c.head_dim, c.dtype = 10, 16, 2, 128, gdn.GDN_BF16
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _attn(batch=2, heads=8, rows=5, max_pages=4, scale=0.1, window=0, q_row_stride=0):
    d = gdn.gdn_attn_desc()
    d.batch, d.num_heads, d.rows, d.max_pages = batch, heads, rows, max_pages
    d.scale, d.window, d.q_row_stride = scale, window, q_row_stride
    return d


def _attend(d, c, **ptrs):
    names = ("q", "k", "v", "table", "cu", "ctx", "o", "lse", "ws", "stream")
    p = {n: PTR * (i + 1) for i, n in enumerate(names)}
    p["stream"] = None
    p.update(ptrs)
    return gdn.library().gdn_paged_attention(ctypes.byref(d) if d is not None else None,
                                             ctypes.byref(c) if c is not None else None, *[p[n] for n in names])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(page_size=12), UNSUPPORTED), (dict(page_size=1), UNSUPPORTED), (dict(page_size=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_kv_heads=3), INVALID),                                            # 8 heads over 3
    (dict(page_stride=4096, row_stride=256), INVALID),                          # a head stride of 0
    (dict(page_stride=4096, row_stride=256, head_stride=64), INVALID),          # below head_dim
    (dict(page_stride=4096, row_stride=260, head_stride=128), INVALID),         # 520 bytes
    (dict(page_stride=-4096, row_stride=256, head_stride=128), INVALID),
    (dict(page_stride=1 << 40, row_stride=256, head_stride=128), INVALID),
])
def test_cache_descriptor_refused(kw, status):
    assert _attend(_attn(), _cache(**kw)) == status
    if kw.get("num_kv_heads") != 3:
        q = _qk()
        q.num_kv_heads = kw.get("num_kv_heads", 2)
        assert _norm(q, _cache(**kw)) in (status, INVALID)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(heads=0), INVALID),
    (dict(heads=7), INVALID), (dict(heads=130), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(window=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q_row_stride=1000), INVALID), (dict(q_row_stride=1028), INVALID),
    (dict(batch=0), OK), (dict(rows=0), OK),                                    # nothing to do: nothing is launched
])
def test_attention_arguments_refused(kw, status):
    assert _attend(_attn(**kw), _cache()) == status


@pytest.mark.parametrize("name", ["q", "k", "v", "table", "cu", "ctx", "o", "ws"])
def test_attention_null_and_misaligned_refused(name):
    assert _attend(_attn(), _cache(), **{name: None}) == INVALID
    assert _attend(_attn(), _cache(), **{name: PTR + 4}) == INVALID


def test_attention_other_refusals():
    assert _attend(None, _cache()) == INVALID
    assert _attend(_attn(), None) == INVALID
    assert _attend(_attn(), _cache(), lse=PTR + 8) == INVALID
    assert _attend(_attn(), _cache(), o=PTR) == INVALID      # in place


def test_workspace_bytes():
    f = gdn.library().gdn_paged_attention_workspace_bytes
    assert f(2, 128, 1) == 0 and f(gdn.GDN_BF16, 96, 1) == 0 and f(gdn.GDN_BF16, 128, -1) == 0
    small, large = f(gdn.GDN_BF16, 128, 1), f(gdn.GDN_BF16, 128, 5000)
    assert small >= 512 and small % 256 == 0 and large % 256 == 0 and large >= small + 32 * 4900
    assert f(gdn.GDN_BF16, 64, 1) < small


def _qk(**kw):
    d = gdn.gdn_qk_desc()
    d.rows, d.num_heads, d.num_kv_heads, d.head_dim, d.rotary_dim, d.dtype = 5, 8, 2, 128, 64, gdn.GDN_BF16
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _norm(d, c, eps=1e-6, **ptrs):
    names = ("q", "k", "v", "pos", "freq", "qw", "kw")
    more = ("slots", "k_pages", "v_pages", "q_out", "k_out")
    p = {n: PTR * (i + 1) for i, n in enumerate(names + more)}
    if c is None:
        p["slots"] = p["k_pages"] = p["v_pages"] = None
    p.update(ptrs)
    return gdn.library().gdn_qk_norm_rope(ctypes.byref(d) if d is not None else None, *[p[n] for n in names], eps,
                                          ctypes.byref(c) if c is not None else None, *[p[n] for n in more], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(num_heads=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(rotary_dim=-16), INVALID),
    (dict(rotary_dim=144), INVALID), (dict(rotary_dim=24), UNSUPPORTED), (dict(rotary_style=2), INVALID),
    (dict(q_row_stride=512), INVALID), (dict(k_row_stride=257), INVALID), (dict(v_row_stride=-8), INVALID),
    (dict(rows=0), OK),
])
def test_norm_rope_arguments_refused(kw, status):
    assert _norm(_qk(**kw), _cache()) == status


def test_norm_rope_other_refusals():
    assert _norm(None, _cache()) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert _norm(_qk(), _cache(), eps=eps) == INVALID
    for name in ("q", "k", "v", "pos", "freq", "slots", "k_pages", "v_pages", "q_out"):
        assert _norm(_qk(), _cache(), **{name: None}) == INVALID
    for name in ("q", "k", "v", "pos", "freq", "qw", "kw", "slots", "k_pages", "v_pages", "q_out", "k_out"):
        assert _norm(_qk(), _cache(), **{name: PTR + 8}) == INVALID
    assert _norm(_qk(), None, k_out=None) == INVALID               # keys would go nowhere
    assert _norm(_qk(), None, slots=PTR) == INVALID                # slots without a cache
    assert _norm(_qk(), _cache(dtype=gdn.GDN_F32)) == INVALID      # another dtype than the rows
    assert _norm(_qk(), _cache(num_kv_heads=4)) == INVALID
    assert _norm(_qk(), _cache(head_dim=64)) == INVALID
    assert _norm(_qk(q_row_stride=2048), _cache(), q_out=PTR) == INVALID       # in place needs packed rows
    assert _norm(_qk(k_row_stride=512), _cache(), k_out=2 * PTR) == INVALID


def test_python_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pos, inv = torch.zeros(4, dtype=torch.int64), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        gdn.qk_norm_rope(x, k, pos, inv)
    c = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    t, cu, ctx = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_paged_attention(x, c, c, t, cu, ctx, x, None, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn._paged_kv(c, c[:, :8])
    with pytest.raises(ValueError):
        gdn._paged_kv(c, c.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        gdn._paged_kv(c, c.float())
    d = gdn._paged_kv(c.transpose(1, 2).contiguous().transpose(1, 2), c.transpose(1, 2).contiguous().transpose(1, 2))
    assert (d.page_stride, d.row_stride, d.head_stride) == (2 * 16 * 128, 128, 16 * 128)
    assert gdn._paged_kv(c, c.clone()).page_stride == 0


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32 + 5])
def test_python_refuses_windows_that_do_not_fit(window):
    with pytest.raises(ValueError):
        gdn._attn_desc(1, 8, 4, 0, 2, window, 1.0)
    assert gdn._attn_desc(1, 8, 4, 0, 2, 2 ** 31 - 1, 1.0).window == 2 ** 31 - 1
