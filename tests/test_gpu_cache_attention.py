"""GPU parity of attention over the paged cache.

Tolerance of a row (u = 2^-24): a score is D products added in fp32, whose order and truncation cost at most 2 u each of
size = scale sum |q_d k_d|, and the argument of 2^x is rounded twice more, 4 u of it; so a weight is off by at most d = (2 D + 8) u size,
relative, plus 2^-21 of the exponential and 2^-11 of its rounding to f16. Sums over n keys add n u. The quotient is then off by
at most (2 d + 2^-11 + 2^-19 + 2 n u) sum p |v| / l, plus weights below f16's range: n keys of at most 2^-31 of the largest weight each,
times the largest |v| that a scale allows; the output's rounding adds 2^-8 of the value. lse: d + 2^-20 + n u, and 4 u of its own size."""
import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32, normal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def cache_of(lengths, H, D, page, seed, spread=0.5, width=None, stacked=False):
    """Pages of quantized normal values under scales that differ from page to page; bytes behind a sequence's end are NaN codes."""
    g = np.random.default_rng(seed)
    need = [max(0, -(-int(n) // page)) for n in lengths]
    pages = sum(need) + 2
    order = g.permutation(pages)
    table = np.full((len(lengths), width or max(need + [1])), 1 << 30, np.int64)
    out = []
    for i in range(2):
        byte = (119 + np.round(spread * g.standard_normal((pages, H)))).astype(np.uint8)
        out.append((plain.encode(g.standard_normal((pages, H, page, D)) * 60), byte))
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        if lengths[b] % page and lengths[b] > 0:
            for i in range(2):
                out[i][0][table[b, n - 1], :, lengths[b] % page:] = 0x7F
    cache = [out[0][0], out[1][0], out[0][1], out[1][1]]
    if stacked:
        both, sc = torch.from_numpy(np.stack(cache[:2], 1)).cuda(), torch.from_numpy(np.stack(cache[2:], 1)).cuda()
        dev = mx.KVCache(both[:, 0], both[:, 1], sc[:, 0], sc[:, 1])
    else:
        dev = mx.KVCache(*(torch.from_numpy(x).cuda() for x in cache))
    return cache, dev, table


def verify(out, lse, q, cache, table, lengths, offsets, scale, window, D):
    ref, rl, mass, size = plain.attention(q.double().cpu().numpy(), cache, table, lengths, offsets, scale, window)
    n = max(int(max(lengths)), 1)
    d = (2 * D + 8) * U * size[:, :, None]
    vmax = 448 * np.nanmax(plain.scale_of(cache[3]))
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((2 * d + 2.0 ** -11 + 2.0 ** -19 + 2 * n * U) * mass + n * 2.0 ** -31 * vmax) + 2.0 ** -133
    got = out.double().cpu().numpy()
    live = np.arange(got.shape[0]) < offsets[-1]
    got, ref, bound, rl, d = got[live], ref[live], bound[live], rl[live], d[live]
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / bound)} at {np.argwhere(bad)[0]}"
    if lse is not None:
        l = lse.double().cpu().numpy()[live]
        ok = np.isfinite(rl)
        assert np.array_equal(l[~ok & ~np.isnan(rl)], rl[~ok & ~np.isnan(rl)]) and np.array_equal(np.isnan(l), np.isnan(rl))
        err = np.abs(l[ok] - rl[ok]) - (d[:, :, 0][ok] + 2.0 ** -20 + n * U + 4 * U * np.abs(rl[ok]))
        assert (err <= 0).all(), err.max()


def check(lengths, rows, Hkv, G, D, page, window=0, seed=0, scale=None, single=False, stacked=False, spread=0.5, sharp=1.0, tail=0):
    cache, dev, table = cache_of(lengths, Hkv, D, page, seed, spread, stacked=stacked)
    offsets = np.concatenate([[0], np.cumsum(rows)])
    q = (normal((int(offsets[-1]) + tail, Hkv * G, D), seed + 1, 0.3) * sharp).cuda()
    out, lse = mx.cache_attention(q, dev, i32(table), i32(lengths), None if single else i32(offsets), scale=scale, window=window,
                                  return_lse=True)
    again = mx.cache_attention(q, dev, i32(table), i32(lengths), None if single else i32(offsets), scale=scale, window=window)
    n = int(offsets[-1])
    assert torch.equal(out[:n].view(torch.int16), again[:n].view(torch.int16))
    assert mx.device_error() == 0
    verify(out, lse, q, cache, table, lengths, offsets, scale or D ** -0.5, window, D)


@pytest.mark.parametrize("Hkv,G,D,page", [(1, 1, 64, 16), (2, 4, 128, 64), (1, 8, 128, 128), (3, 5, 64, 32), (2, 16, 128, 16), (1, 40, 64, 64),
                                          (2, 12, 128, 32)])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_single_tokens(Hkv, G, D, page, window):
    lengths = [1, 2, 15, 16, 17, 63, 64, 65, 0, 128, 300, 1025]
    check(lengths, [1] * len(lengths), Hkv, G, D, page, window, seed=G, single=True)


@pytest.mark.parametrize("lengths", [[1], [5000], [20000, 3, 700], [64] * 130, [0, 0, 0], [9000] * 3])
def test_splits_and_batches(lengths):
    check(lengths, [1] * len(lengths), 2, 4, 128, 64, seed=len(lengths), single=True)


@pytest.mark.parametrize("Hkv,G,D,page", [(1, 1, 64, 16), (2, 4, 128, 64), (1, 8, 128, 128), (3, 3, 64, 32), (1, 6, 128, 16)])
@pytest.mark.parametrize("window", [0, 7, 200])
def test_ragged_rows(Hkv, G, D, page, window):
    rows = [1, 3, 0, 70, 2, 1, 129, 300, 5]
    before = [0, 40, 9, 0, 500, 0, 33, 100, 2000]
    check([a + n for a, n in zip(before, rows)], rows, Hkv, G, D, page, window, seed=page, tail=3, stacked=True)


@pytest.mark.parametrize("D,G", [(128, 4), (64, 1), (128, 7)])
def test_prompts(D, G):
    rows = [513, 256, 255, 1, 1000]
    check(rows, rows, 1, G, D, 64, seed=D + G)
    check([n + 777 for n in rows], rows, 1, G, D, 16, window=300, seed=G)


def test_rows_without_keys():
    """Fewer tokens than rows, none, negative: zeros and -inf."""
    check([2, 0, -5, 60], [4, 3, 2, 70], 1, 4, 128, 16)
    check([0, 3, -1], [1, 1, 1], 2, 2, 64, 32, single=True)


@pytest.mark.parametrize("single", [True, False])
def test_page_scales_that_differ_widely(single):
    rows = [1, 1, 1] if single else [40, 3, 90]
    for spread, seed in ((6.0, 1), (0.0, 2)):
        check([500, 90, 1300], rows, 2, 4, 128, 32, spread=spread, seed=seed, single=single)


@pytest.mark.parametrize("single", [True, False])
def test_sharp_and_flat_scores(single):
    rows = [1, 1] if single else [100, 260]
    for sharp, scale in ((20.0, None), (0.01, None), (1.0, 2.0), (2.0 ** -60, None)):
        check([900, 300], rows, 2, 4, 128, 64, sharp=sharp, scale=scale, seed=3, single=single)


@pytest.mark.parametrize("rows", [1, 80])
def test_nan_pages_and_bad_pages_reach_only_the_rows_that_see_them(rows):
    """A page whose scale says NaN, one outside the pool, one behind the table."""
    Hkv, G, D, page = 2, 4, 128, 16
    lengths, offsets = np.array([200, 200, 200, 200]), np.arange(5) * rows
    cache, dev, table = cache_of(lengths, Hkv, D, page, 1)
    cache[2][table[0, 11], 0] = 255           # the last full page's keys, head 0
    cache[3][table[1, 10], 1] = 255           # values, head 1
    table[2, 9] = 1 << 29
    dev = mx.KVCache(*(torch.from_numpy(x).cuda() for x in cache))
    q = normal((4 * rows, Hkv * G, D), 2).cuda()
    mx.device_error()
    for t in (table, table[:, :12]):          # then without the last page's column
        out, lse = mx.cache_attention(q, dev, i32(t), i32(lengths), i32(offsets), return_lse=True)
        assert mx.device_error() == 4
        verify(out, lse, q, cache, t, lengths, offsets, D ** -0.5, 0, D)


@pytest.mark.parametrize("rows", [1, 100])
def test_queries_of_nan_concern_their_own_row(rows):
    cache, dev, table = cache_of([300], 1, 128, 64, 5)
    q = normal((rows, 4, 128), 3).cuda()
    want = mx.cache_attention(q, dev, i32(table), i32([300]), i32([0, rows]))
    q[rows - 1, 2, 7] = float("nan")
    got = mx.cache_attention(q, dev, i32(table), i32([300]), i32([0, rows]))
    assert got[rows - 1, 2].isnan().all()
    got[rows - 1, 2] = want[rows - 1, 2]
    assert torch.equal(got, want)


def test_rows_behind_the_last_sequence_and_strided_tensors():
    """q and out as views of wider tensors; what lies between and behind stays."""
    cache, dev, table = cache_of([100, 50], 2, 64, 32, 6)
    wide = normal((30, 10, 64), 1).cuda()
    q = wide[:, 2:8]
    out = torch.full((30, 9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    offsets = np.array([0, 20, 23])
    got = mx.cache_attention(q, dev, i32(table), i32([100, 50]), i32(offsets), out=out[:, 1:7])
    verify(got, None, q, cache, table, np.array([100, 50]), offsets, 64 ** -0.5, 0, 64)
    assert (out[23:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 7:] == 7).all()


def test_offsets_past_the_tensors_are_cut():
    """Row offsets that run past the rows, or backwards, touch nothing outside."""
    cache, dev, table = cache_of([100, 50, 60], 1, 64, 16, 7)
    q = normal((12, 4, 64), 1).cuda()
    big = torch.full((40, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    for offsets in ([0, 4, 1 << 30, 8], [-5, 4, 2, 50], [20, 30, 40, 50]):
        mx.cache_attention(q, dev, i32(table), i32([100, 50, 60]), i32(offsets), out=big[10:22])
        mx.cache_append(q[:, :1], q[:, :1], dev, i32(table), i32([100, 50, 60]), i32(offsets), q=q, out=big[10:22])
        assert (big[:10] == 5).all() and (big[22:] == 5).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [1, 150])
def test_captured_twice_with_lengths_that_change(rows):
    """Two graphs of the same call replayed in turn on two streams while lengths grow between replays."""
    Hkv, G, D, page, B = 2, 4, 128, 64, 3
    lengths = np.array([700, 333, 1500])
    cache, dev, table = cache_of(lengths, Hkv, D, page, 8)
    offsets = None if rows == 1 else i32(np.arange(B + 1) * rows)
    q = [normal((B * rows, Hkv * G, D), i).cuda() for i in range(2)]
    lens = i32(lengths - 40)
    tab = i32(table)
    graphs, outs = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.cache_attention(x, dev, tab, lens, offsets))
        graphs.append(g)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        torch.cuda.synchronize()
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, o in zip(q, outs):
            assert torch.equal(o, mx.cache_attention(x, dev, tab, lens, offsets))
        lens += 40


def test_a_layers_steps():
    """Prompts, then decoding, as a sampler runs them: append with rotation, attention; against the same in fp64 on the
    codes that the cache then holds, and the codes against their definition."""
    Hkv, G, D, page, B = 2, 3, 64, 16, 4
    rows = np.array([37, 5, 64, 1])
    need = 8
    cache = mx.cache_create(B * need, Hkv, D, page)
    table = np.random.default_rng(1).permutation(B * need).reshape(B, need)
    tab = mx.rope_table(128, D, base=1e4)
    codes = [to_np(cache.k).copy(), to_np(cache.v).copy()]
    byte = [to_np(cache.k_scale).copy(), to_np(cache.v_scale).copy()]
    lengths = rows.copy()
    for step in range(12):
        offsets = np.concatenate([[0], np.cumsum(rows)])
        T = int(offsets[-1])
        q, k, v = normal((T, Hkv * G, D), step).cuda(), normal((T, Hkv, D), 50 + step), normal((T, Hkv, D), 90 + step)
        where = (cache, i32(table), i32(lengths), i32(offsets) if step < 2 else None)
        qr = mx.cache_append(k.cuda(), v.cuda(), *where, q=q, table=tab)
        out, lse = mx.cache_attention(qr, *where, return_lse=True)
        pos = np.concatenate([l - n + np.arange(n) for l, n in zip(lengths, rows)])
        kr = plain.rope(k.double().numpy(), to_np(tab), pos, False)
        for i, x in enumerate((kr, v.double().numpy())):
            codes[i], byte[i] = plain.append((codes[i], byte[i]), x, table, lengths, offsets)
            assert np.array_equal(to_np(cache[i]), codes[i]) and np.array_equal(to_np(cache[2 + i]), byte[i])
        assert torch.equal(qr, mx.rope(q, tab, i32(pos)))
        verify(out, lse, qr, [codes[0], codes[1], byte[0], byte[1]], table, lengths, offsets, D ** -0.5, 0, D)
        rows = np.ones(B, np.int64)
        lengths = lengths + 1


@pytest.mark.parametrize("G,rows", [(1, [32, 33, 47, 48, 49, 50]), (4, [8, 9, 12, 13]), (5, [9, 10]), (12, [4, 5])])
def test_rows_around_the_kernels_border(G, rows):
    """Sequences whose rows per key head are just below, at and above the number that one kernel hands to the other."""
    check([n + before for n, before in zip(rows, [0, 300, 7, 1100, 64, 2])], rows, 2, G, 128, 32, seed=G, tail=1)
    check([n + 90 for n in rows], rows, 1, G, 64, 16, window=33, seed=G)
