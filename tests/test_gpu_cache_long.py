"""The cache and attention where offsets pass 32 bits, lengths are long and batches wide, and where waits run out."""
import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32, normal
from test_gpu_cache_attention import cache_of, check, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 70])
def test_pages_past_four_gigabytes(rows):
    """A pool of 6 GB a tensor, its last pages in use: appended to and attended."""
    H, D, page, pages = 2, 128, 64, 380000
    cache = mx.cache_create(1, H, D, page)
    pool = [torch.empty((pages, H, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, H), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = mx.KVCache(pool[0], pool[1], scales[0], scales[1])
    ids = pages - 1 - np.array([[0, 3, 1], [5, 2, 4]])
    lengths, before = np.array([150, 100]), np.array([150 - rows, 100 - rows])
    small = [np.zeros((6, H, page, D), np.uint8), np.zeros((6, H, page, D), np.uint8)]
    byte = [np.zeros((6, H), np.uint8), np.zeros((6, H), np.uint8)]
    table = pages - 1 - ids
    for n, total in ((before, before), (np.array([rows, rows]), lengths)):
        offsets = np.concatenate([[0], np.cumsum(n)])
        k, v = normal((int(offsets[-1]), H, D), 1), normal((int(offsets[-1]), H, D), 2)
        mx.cache_append(k.cuda(), v.cuda(), cache, i32(ids), i32(total), i32(offsets))
        for i, x in enumerate((k, v)):
            small[i], byte[i] = plain.append((small[i], byte[i]), x.double().numpy(), table, total, offsets)
    for i in range(2):
        top = to_np(cache[i][pages - 6:])[::-1]
        used = [(b, p) for b in range(2) for p in range(-(-lengths[b] // page))]
        for b, p in used:
            n = min(page, lengths[b] - p * page)
            assert np.array_equal(top[table[b, p]][:, :n], small[i][table[b, p]][:, :n])
    q = normal((2 * rows, 4 * H, D), 3).cuda()
    out, lse = mx.cache_attention(q, cache, i32(ids), i32(lengths), i32(np.arange(3) * rows), return_lse=True)
    verify(out, lse, q, [small[0], small[1], byte[0], byte[1]], table, lengths, np.arange(3) * rows, D ** -0.5, 0, D)


def test_a_long_sequence():
    check([150001], [1], 1, 8, 128, 128, seed=1, single=True)
    check([60000], [100], 1, 4, 64, 16, seed=2)
    check([60000], [100], 1, 4, 64, 16, window=5000, seed=2)


def test_many_sequences():
    """More sequences than threads of any block: singles, and prompts among them."""
    g = np.random.default_rng(3)
    check(g.integers(0, 90, 700), [1] * 700, 1, 4, 64, 16, seed=4, single=True)
    rows = g.integers(0, 3, 400)
    rows[::50] = 40
    check(g.integers(0, 60, 400) + rows, rows, 2, 2, 64, 16, seed=5)


def test_units_cut_in_many_ways():
    """Item counts and lengths that put the cuts between blocks at every place of a unit."""
    for n, before, Hkv, G in ((9, 4000, 1, 8), (256, 0, 3, 1), (257, 900, 2, 1), (300, 1, 5, 4), (65, 7777, 4, 4)):
        check([n + before, n], [n, n], Hkv, G, 128, 32, seed=n)


@pytest.mark.parametrize("D", [64, 128])
def test_short_deadlines(D):
    """Under deadlines down to 1 ns a wait may run out (this kernel's mostly end within their first try): then its bit is set and a row
    is its value or what was there; otherwise all is as ever. The next call is right."""
    lengths, rows = np.array([9000, 3000]), np.array([700, 900])
    cache, dev, table = cache_of(lengths, 2, D, 64, 3)
    q = normal((1600, 8, D), 1).cuda()
    where = (dev, i32(table), i32(lengths), i32([0, 700, 1600]))
    want = mx.cache_attention(q, *where)
    assert mx.device_error() == 0
    try:
        for ns in (1, 1, 5000, 20000, 50000, 100000, 200000) * 2:
            out = torch.full_like(want, -7.0)
            mx.set_wait_timeout_ns(ns)
            mx.cache_attention(q, *where, out=out)
            torch.cuda.synchronize()
            bits = mx.device_error()
            assert bits in (0, 1)
            same, none = (out == want).all(-1), (out == -7.0).all(-1)
            assert (same | none).all()
            if not bits:
                assert torch.equal(out, want)
    finally:
        mx.set_wait_timeout_ns(0)
    assert torch.equal(mx.cache_attention(q, *where), want)


def test_offsets_that_name_rows_twice():
    """More rows than there are: reported or not, nothing outside is touched and the next call is right."""
    cache, dev, table = cache_of([200] * 60, 1, 64, 16, 7)
    q = normal((100, 4, 64), 1).cuda()
    out = torch.full((120, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.device_error()
    offsets = [0, 100] * 30 + [0]
    mx.cache_attention(q, dev, i32(table), i32([200] * 60), i32(offsets), out=out[10:110])
    torch.cuda.synchronize()
    assert mx.device_error() in (0, 2)
    assert (out[:10] == 5).all() and (out[110:] == 5).all()
    check([200], [100], 1, 4, 64, 16)


def test_two_streams_at_once():
    """Calls of every kind in flight on two streams at the same time give what they give alone."""
    cache, dev, table = cache_of([3000, 900, 40], 2, 128, 64, 9)
    lens = i32([3000, 900, 40])
    q = normal((600, 8, 128), 1).cuda()
    one = q[:3].contiguous()
    offsets = i32([0, 500, 599, 600])
    want = [mx.cache_attention(q, dev, i32(table), lens, offsets), mx.cache_attention(one, dev, i32(table), lens)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    t = i32(table)
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((mx.cache_attention(q, dev, t, lens, offsets), mx.cache_attention(one, dev, t, lens)))
    torch.cuda.synchronize()
    for pairs in got:
        for a, b in pairs:
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
