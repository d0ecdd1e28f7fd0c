"""Sizes of the attention's workspace (host code only, no GPU needed)."""
import ctypes

import pytest

from mxfp8_block_scaled_07_b200 import build as mxbuild, mx
from test_abi_cache import A, BAD_BATCHES, BIG, batch


@pytest.fixture(scope="module")
def sizes():
    mxbuild.build()
    lib = mx.lib()
    return lambda q_heads=8, **kw: lib.mx_cache_attention_batch_bytes(ctypes.byref(batch(mx, **{**dict(sequences=4, rows=4, row_offsets=None), **kw})), q_heads)


def test_without_row_offsets(sizes):
    """Only the parts of few rows: 8 MB at most, next to nothing for one short sequence, less for narrow tables than for wide ones."""
    wide = dict(head_dim=128, heads=8, k_stride=1 << 20, v_stride=1 << 20, ks_stride=8, vs_stride=8, ld_table=1 << 20, width=1 << 20)
    assert 0 < sizes(q_heads=32, **wide) <= 4.1e6 and 4.1e6 < sizes(q_heads=128, **wide) <= 8.1e6
    assert 0 < sizes(q_heads=32, **{**wide, "sequences": 1, "rows": 1, "width": 17}) < 1e6
    assert sizes(width=1) <= sizes(width=2) <= sizes(width=40, ld_table=40)
    assert sizes(sequences=1 << 20, rows=1 << 20) <= 8.1e6


def test_with_row_offsets(sizes):
    """Sequences with many rows: more, and no more than for any batch of such sizes; none where the rows cannot make any."""
    some = dict(head_dim=128, heads=8, k_stride=1 << 20, v_stride=1 << 20, ks_stride=8, vs_stride=8, row_offsets=A, width=4000, ld_table=4000)
    whole = mx.lib().mx_cache_attention_workspace_bytes
    for rows in (1, 12, 13, 100, 5000, 100000):
        for heads in (8, 32, 64):
            assert 0 < sizes(q_heads=heads, rows=rows, **some) <= whole(128, rows, heads)
            assert sizes(q_heads=heads, rows=rows, **some) <= 8.1e6 + 43e6 + 2 * rows * heads
    assert sizes(q_heads=32, rows=12, **some) <= 8.1e6 < 4e7 < sizes(q_heads=32, rows=5000, **some)
    # Two pages of 64: 10 items of 8 heads, 6 units of cost each, 8 a block at least; 4 sequences of 8 heads and 3 tiles, 4 steps each, 2 a block.
    assert sizes(q_heads=32, rows=100, **{**some, "width": 2}) <= (60 * 2 * 256 + 192 * 2 * 16) * 131 * 4 + 4096


def test_refusals(sizes):
    """What the call refuses has no size; a batch without work needs none."""
    for kw, _ in BAD_BATCHES:
        if not {"k", "v", "v_scale", "lengths", "page_table", "row_offsets", "k_stride", "vs_stride", "ld_table", "v_stride"} & set(kw):
            assert sizes(**{**dict(row_offsets=A), **kw}) == -1, kw
    assert sizes(row_offsets=None, rows=3) == -1 and sizes(q_heads=0) == -1 and sizes(q_heads=7) == -1 and sizes(q_heads=4098) == -1
    assert sizes(row_offsets=A, rows=BIG - 1) == -1
    assert sizes(rows=0, sequences=0) == 0 and sizes(row_offsets=A, rows=0) == 0
    assert mx.lib().mx_cache_attention_batch_bytes(None, 4) == -1
