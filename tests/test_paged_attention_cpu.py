"""Paged attention's host-side parts that need no device."""
import os
import random
import re

import numpy as np
import pytest
import torch


import gated_deltanet_state_tail_b200 as gdn


def test_split_table_entries_outside_the_call_are_not_merged():
    """Whatever bytes a call that gave up leaves in the table of split units, the merging kernel reads parts and writes
    rows of this call only."""
    rng = random.Random(5)
    words = [-2 ** 31, -1, 0, 1, 2, 7, 31, 127, 147, 148, 255, 4096, 0x7F7F7F7F, 2 ** 31 - 1]
    taken = 0
    for _ in range(20000):
        entry = [rng.choice(words) if rng.random() < 0.5 else rng.randint(-3, 160) for _ in range(5)]
        index, parts = rng.randrange(148), 148
        toks, rows, heads = rng.choice([1, 2, 16, 256]), rng.choice([1, 5, 300, 2 ** 31 - 1]), rng.choice([1, 3, 8])
        if gdn.gdn_selftest_split_entry(entry, index, parts, toks, rows, heads):
            last, _, row0, n, head = entry
            assert index < last < parts and 0 < n <= toks and 0 <= row0 and row0 + n <= rows and 0 <= head < heads
            taken += 1
    assert taken > 20
    assert gdn.gdn_selftest_split_entry([148 - 1, 1, 44, 256, 2], 146, 148, 256, 300, 3)
    assert not gdn.gdn_selftest_split_entry([-1, 0, 0, 1, 0], 0, 148, 256, 300, 3)          # no unit
    assert not gdn.gdn_selftest_split_entry([3, 0, 0, 1, 0], 3, 148, 256, 300, 3)           # one part is not a split
    assert not gdn.gdn_selftest_split_entry([148, 0, 0, 1, 0], 3, 148, 256, 300, 3)
    assert not gdn.gdn_selftest_split_entry([5, 0, 2 ** 31 - 1, 256, 0], 3, 148, 256, 2 ** 31 - 1, 3)   # past 32 bits


def test_expanded_rows_are_refused():
    """A stride of 0 is the descriptors' word for packed rows: one row expanded to many would be read past its end."""
    x = torch.zeros(8, 128)
    for rows in (2, 4096):
        y = x[None].expand(rows, 8, 128)
        with pytest.raises(ValueError, match="q must not"):
            gdn._row_stride(y.shape, y.stride(), "q")
    one = x[None].expand(1, 8, 128)
    assert gdn._row_stride(one.shape, one.stride(), "q") == 0
    wide = torch.zeros(4, 12, 128)[:, :8]
    assert gdn._row_stride(wide.shape, wide.stride(), "q") == 12 * 128


def test_expanded_rows_of_a_plan_call_are_refused():
    x = torch.zeros(4, 128)
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)[None].expand(50, 4, 128)
        with pytest.raises(ValueError, match="expanded"):
            gdn.row_stride_of(y, y)
        with pytest.raises(ValueError, match="expanded"):
            gdn.row_stride_of(torch.zeros(50, 4, 128, dtype=dtype), y)
    assert gdn.row_stride_of(x[None], None, x[None]) == 0
    wide = torch.zeros(5, 3, 4, 128)
    assert gdn.row_stride_of(wide[:, 0], wide[:, 1], wide[:, 2]) == 3 * 4 * 128


@pytest.mark.parametrize("shape", [(3, 16, 2, 128), (3, 1, 1, 128), (1, 16, 1, 128), (1, 1, 2, 128), (3, 16, 1, 128)])
def test_expanded_caches_are_refused(shape):
    row = torch.zeros(128).expand(*shape)
    with pytest.raises(ValueError, match="expanded"):
        gdn._paged_kv(row, row)
    pages = torch.zeros(16, 2, 128)[None].expand(3, 16, 2, 128)
    with pytest.raises(ValueError, match="expanded"):
        gdn._paged_kv(pages, pages)
    assert gdn._paged_kv(torch.zeros(shape), torch.zeros(shape)).page_stride == 0


def test_refusals_name_misaligned_tensors():
    x = torch.zeros(8, dtype=torch.int64)
    x = x[(-x.data_ptr() // 8) % 2:]
    with pytest.raises(gdn.GdnError, match="positions, slots must start on a 16-byte") as e:
        gdn._refused(gdn.GDN_ERR_INVALID_ARG, "call", q=x, positions=x[1:], k_out=None, slots=x[3:4])
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    for status, tensors in ((gdn.GDN_ERR_INVALID_ARG, dict(q=x)), (gdn.GDN_ERR_CUDA, dict(q=x[1:]))):
        with pytest.raises(gdn.GdnError) as e:
            gdn._refused(status, "call", **tensors)
        assert "boundary" not in str(e.value) and e.value.status == status


def test_polynomial_exponential():
    """2^f on [-1/2, 1/2] by the kernel's coefficients, in fp32 with fused multiply-adds (an fp64 product of two fp32
    values is exact), against fp64: the error that the kernel states."""
    path = os.path.join(os.path.dirname(gdn.__file__), "csrc", "gdn_attn_tc.cu")
    body = open(path).read().split("float2 ex2_poly(Pair y)")[1].split("const float2 e =")[0]
    c = [np.float32(x) for x in re.findall(r"pair\(([0-9.]+)f, \1f\)", body.split("Pair p =")[1])]
    assert len(c) == 6 and c[-1] == 1
    f = np.linspace(-0.5, 0.5, 200001).astype(np.float32)
    p = np.full_like(f, c[0])
    for x in c[1:]:
        p = (p.astype(np.float64) * f + np.float64(x)).astype(np.float32)
    want = np.exp2(f.astype(np.float64))
    assert float(np.abs(p / want - 1).max()) <= 4.9e-7
    assert p[np.flatnonzero(f == 0)[0]] == 1
