"""Attention over pages whose value scales lie far apart: a row's precision hangs on the keys that it sees and on nothing else.

The bound is a row's own. With u = 2^-24, d = (2 D + 8) u size the error of a score's power of two (see test_gpu_cache_attention) and n keys, the
quotient is off by (2 d + 2^-11 + 2^-19 + 2 n u) sum p |v| / l. Weights are rounded to f16 relative to the row's largest product of weight and
value scale, which stands at 2^6.5 at least: what lies below f16's normal numbers is off by 2^-25, less than 2^-31 of that product, for each of
n keys, times the largest code, 448. The output's rounding adds 2^-8 of the value. lse: d + 2^-20 + n u, and 4 u of its own size."""
import numpy as np
import pytest
import torch

import plain_cache as plain
from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def reach(q, cache, page_table, lengths, offsets, scale, window, lse):
    """max_j p_j 448 2^e_j / l over the keys that a row sees, [T, Hq]."""
    k_codes, _, ks, vs = cache
    T, Hq, D = q.shape
    Hkv, page = k_codes.shape[1], k_codes.shape[2]
    out = np.zeros((T, Hq))
    for b in range(len(lengths)):
        r0, n, total = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(lengths[b])
        at = page_table[b, :-(-total // page)]
        i, j = total - n + np.arange(n)[:, None], np.arange(total)[None, :]
        seen = (j <= i) & ((j > i - window) if window > 0 else True)
        for h in range(Hkv):
            k = (plain.decode(k_codes[at, h]) * plain.scale_of(ks[at, h])[:, None, None]).reshape(-1, D)[:total]
            e = np.repeat(plain.scale_of(vs[at, h]), page)[:total]
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = scale * np.einsum("rd,kd->rk", q[r0:r0 + n, g], k)
                p = np.where(seen, np.exp(np.minimum(z - lse[r0:r0 + n, g, None], 0.0)), 0.0)
                out[r0:r0 + n, g] = (p * e).max(1) * 448
    return out


def check(lengths, rows, Hkv, G, D, page, scores, v_bytes, window=0, seed=0, single=False):
    """Keys whose score with every query is about scores(position) (natural log), pages of values under v_bytes(page of its sequence, heads)."""
    g = np.random.default_rng(seed)
    lengths, offsets = np.asarray(lengths), np.concatenate([[0], np.cumsum(rows)])
    T, B = int(offsets[-1]), len(lengths)
    need = [-(-int(n) // page) for n in lengths]
    pages = sum(need) + 1
    order = g.permutation(pages)
    table = np.zeros((B, max(need)), np.int64)
    k, v = (np.zeros((pages, Hkv, page, D), np.uint8) for _ in range(2))
    ks, vs = (np.full((pages, Hkv), 100, np.uint8) for _ in range(2))
    # q: ones in the first half of the features, small noise behind; keys: a constant there, noise behind.
    q = np.concatenate([np.ones((T, Hkv * G, D // 2)), g.standard_normal((T, Hkv * G, D // 2)) * 0.25], 2)
    q = torch.from_numpy(q).to(torch.bfloat16)
    scale = D ** -0.5
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        for p in range(n):
            t = scores(p * page + np.arange(page))[None, :, None] / scale / (D // 2)
            kk = np.broadcast_to(t, (Hkv, page, D)).copy()
            kk[..., D // 2:] = g.standard_normal((Hkv, page, D // 2)) * 0.25
            byte = 127 - 8 + int(np.ceil(np.log2(np.abs(kk).max())))
            k[table[b, p]], ks[table[b, p]] = plain.encode(np.ldexp(kk, 127 - byte)), byte
            v[table[b, p]] = plain.encode(g.standard_normal((Hkv, page, D)) * 100)
            vs[table[b, p]] = v_bytes(p, np.arange(Hkv), g)
    cache = (k, v, ks, vs)
    dev = mx.KVCache(*(torch.from_numpy(x).cuda() for x in cache))
    out, lse = mx.cache_attention(q.cuda(), dev, i32(table), i32(lengths), None if single else i32(offsets), window=window, return_lse=True)
    assert mx.device_error() == 0
    q = q.double().numpy()
    ref, rl, mass, size = plain.attention(q, cache, table, lengths, offsets, scale, window)
    n = int(lengths.max())
    d = (2 * D + 8) * U * size
    most = reach(q, cache, table, lengths, offsets, scale, window, rl)
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((2 * d[..., None] + 2.0 ** -11 + 2.0 ** -19 + 2 * n * U) * mass + n * 2.0 ** -31 * most[..., None]) + 2.0 ** -133
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= bound).all(), f"{(~(err <= bound)).sum()} of {err.size} off, worst {np.nanmax(err / bound)} at {np.argwhere(~(err <= bound))[0]}"
    err = np.abs(lse.double().cpu().numpy() - rl) - (d + 2.0 ** -20 + n * U + 4 * U * np.abs(rl))
    assert (err <= 0).all(), err.max()


# Sequences with few rows per key head, with many, and single tokens without offsets.
FORMS = {"few": ([150, 64, 130], [40, 12, 48], 2, 1, False), "many": ([150, 128, 700], [150, 128, 500], 1, 2, False),
         "single": ([150, 64, 700], [1, 1, 1], 2, 5, True), "wide": ([150, 700], [1, 1], 1, 24, True)}
APART = [20, 25, 28, 32, 45, 58, 90, 120]


def run(form, D, page, scores, v_bytes, **kw):
    lengths, rows, Hkv, G, single = FORMS[form]
    check(lengths, rows, Hkv, G, D, page, scores, v_bytes, single=single, **kw)


@pytest.mark.parametrize("apart", APART)
@pytest.mark.parametrize("form", ["few", "many"])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
def test_pages_that_a_row_does_not_see_yet(form, apart, D, page):
    """Values grow from page to page: what stands behind a row's position takes nothing from it."""
    run(form, D, page, lambda j: 0.1 * np.cos(j), lambda p, h, g: np.minimum(100 + apart * (p % 2) + h, 246))


@pytest.mark.parametrize("apart", APART)
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D,page", [(128, 32), (64, 64)])
def test_pages_that_a_row_sees_without_weight(form, apart, D, page):
    """Every third page's values are far larger, but its keys have no weight to speak of."""
    run(form, D, page, lambda j: np.where(j // page % 3 == 1, -60.0, 30.0) + np.cos(j), lambda p, h, g: np.minimum(100 + apart * (p % 3 == 1) + h, 246))


@pytest.mark.parametrize("apart", APART)
@pytest.mark.parametrize("form", ["few", "many", "single"])
def test_pages_in_front_of_the_window(form, apart):
    run(form, 128, 16, lambda j: 0.1 * np.cos(j), lambda p, h, g: np.where(p % 4 == 3, 100 + apart, 100), window=20)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_there_is(form, D):
    """Scales from 2^-127 to 2^119 in random order, scores between -90 and 90, so that weights, values, both or neither decide a row."""
    for seed in range(3):
        run(form, D, 16, lambda j: 90 * np.cos(j // 16 * (seed + 2.3)), lambda p, h, g: g.integers(0, 247, h.size), seed=seed)
        run(form, D, 32, lambda j: 80.0 - 160 * (j % 2), lambda p, h, g: g.choice([0, 246], h.size), seed=seed)


@pytest.mark.parametrize("window", [0, 3000])
@pytest.mark.parametrize("rows,G", [(1, 4), (30, 1), (90, 2)])
def test_parts_of_long_sequences(rows, G, window):
    """Sequences whose keys are shared among many blocks, with a scale of its own in every page."""
    check([9000, 2500], [rows, rows], 1, G, 128, 64, lambda j: 40 * np.cos(j // 64 * 1.7), lambda p, h, g: g.integers(0, 247, h.size), window=window,
          single=rows == 1)
