"""GPU parity of the appended cache: codes and scale bytes are those of the fp64 definition, byte for byte; rotated queries within
three fp32 steps (the sum of two products) and half a BF16 step."""
import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu


def setup(lengths, rows, H, D, page, seed, width=None, stacked=False):
    """A cache of garbage, a page table over shuffled pages, row offsets of the rows of every sequence."""
    g = np.random.default_rng(seed)
    need = [max(0, -(-int(n) // page)) for n in lengths]
    width = width or max(need + [1])
    pages = sum(need) + 3
    order = g.permutation(pages)
    table = np.full((len(lengths), width), -7, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    offsets = np.concatenate([[0], np.cumsum(rows)])
    codes = [g.integers(0, 256, (pages, H, page, D)).astype(np.uint8) for _ in range(2)]
    codes = [np.where((c & 127) == 127, c - 1, c).astype(np.uint8) for c in codes]
    byte = [g.integers(110, 130, (pages, H)).astype(np.uint8) for _ in range(2)]
    if stacked:
        both = torch.from_numpy(np.stack(codes, 1)).cuda()
        sc = torch.from_numpy(np.stack(byte, 1)).cuda()
        cache = mx.KVCache(both[:, 0], both[:, 1], sc[:, 0], sc[:, 1])
    else:
        cache = mx.KVCache(*(torch.from_numpy(x).cuda() for x in (*codes, *byte)))
    return codes, byte, cache, table, offsets


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def normal(shape, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(sigma * torch.randn(shape[:-1] + (1,), generator=g))).to(torch.bfloat16)


def check(lengths, rows, H, D, page, rot=None, interleaved=False, Hq=0, seed=0, single=False, stacked=False, positions=4096, tail=0, special=None):
    codes, byte, cache, table, offsets = setup(lengths, rows, H, D, page, seed, stacked=stacked)
    T = int(offsets[-1]) + tail
    k, v = normal((T, H, D), seed + 1), normal((T, H, D), seed + 2)
    if special is not None:
        special(k, v)
    tab = plain.table(positions, plain.frequencies(rot)) if rot else None
    lengths = np.asarray(lengths)
    pos = np.full(T, -1)
    for b, n in enumerate(rows):
        pos[offsets[b]:offsets[b] + n] = lengths[b] - n + np.arange(n)
    kr = plain.rope(k.double().numpy(), tab, pos, interleaved) if rot else k.double().numpy()
    q = normal((T, Hq, D), seed + 3) if Hq else None
    got = mx.cache_append(k.cuda(), v.cuda(), cache, i32(table), i32(lengths), None if single else i32(offsets),
                          q=q.cuda() if Hq else None, table=torch.from_numpy(tab).cuda() if rot else None, interleaved=interleaved)
    for x, code, b8, c_d, s_d in ((kr, codes[0], byte[0], cache.k, cache.k_scale), (v.double().numpy(), codes[1], byte[1], cache.v, cache.v_scale)):
        want_c, want_s = plain.append((code, b8), x, table, lengths, offsets)
        assert np.array_equal(to_np(s_d), want_s)
        bad = np.argwhere(to_np(c_d) != want_c)
        assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0]}"
    if Hq:
        want = plain.rope(q.double().numpy(), tab, pos, interleaved) if rot else np.where(pos[:, None, None] >= 0, q.double().numpy(), 0)
        live = np.zeros(T, bool)
        live[:int(offsets[-1])] = True
        err = np.abs(got.double().cpu().numpy() - want)[live]
        assert (err <= (2.0 ** -8 + 3 * 2.0 ** -24) * np.abs(want[live]) + 2.0 ** -133).all()
    else:
        assert got is None


@pytest.mark.parametrize("H,D,page", [(1, 64, 16), (2, 128, 16), (4, 64, 128), (3, 128, 32), (8, 128, 64), (2, 128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_single_tokens(H, D, page, interleaved):
    lengths = [1, 2, page, page + 1, 2 * page, 0, 3 * page - 1, 700]
    check(lengths, [1] * 8, H, D, page, rot=D, interleaved=interleaved, Hq=2 * H, single=True, seed=H)
    check(lengths, [1] * 8, H, D, page, rot=16, interleaved=interleaved, Hq=5 * H, single=False, seed=H)


@pytest.mark.parametrize("H,D,page", [(1, 64, 16), (2, 128, 16), (4, 64, 128), (3, 128, 32), (8, 128, 64), (2, 128, 128)])
def test_ragged_prompts(H, D, page):
    rows = [5, 0, 1, 3 * page, page + 1, 200, 2, 130]
    before = [0, 9, page - 1, 0, page // 2, 1, 3 * page, page]
    check([a + n for a, n in zip(before, rows)], rows, H, D, page, rot=D // 2, Hq=3 * H, seed=D + page)
    check([a + n for a, n in zip(before, rows)], rows, H, D, page, rot=D, interleaved=True, seed=D, tail=7, stacked=True)
    check([a + n for a, n in zip(before, rows)], rows, H, D, page, seed=1, Hq=H)


def test_many_sequences():
    g = np.random.default_rng(5)
    rows = g.integers(0, 4, 100)
    before = g.integers(0, 90, 100)
    check(before + rows, rows, 2, 64, 16, rot=64, Hq=2, seed=8)


def test_sequences_shorter_than_their_rows():
    """Padding: fewer tokens than rows, none, a negative length."""
    check([2, 0, -3, 20], [4, 2, 1, 3], 2, 128, 16, rot=128, Hq=4, seed=2)
    check([0, -1, 5], [1, 1, 1], 2, 64, 32, rot=64, Hq=2, single=True, seed=2)


def test_zeros_tiny_and_huge_values():
    def special(k, v):
        k[0] = 0
        v[0] = -0.0
        k[1] *= 2.0 ** -120
        v[1] *= 2.0 ** 100
        v[2] = 2.0 ** -133
        k[3] = torch.finfo(torch.bfloat16).max / 4
        v[4] = 448.0
        v[5] = 449.0
        v[6] = 500.0
    check([1] * 8, [1] * 8, 2, 64, 16, rot=64, single=True, special=special)
    check([8], [8], 2, 64, 16, rot=64, special=special)


def test_nan_and_infinity_take_the_block_out_until_it_is_begun_anew():
    page, H, D = 16, 2, 64
    cache = mx.cache_create(4, H, D, page)
    table = i32([[2, 1]])
    k = normal((1, H, D), 1).cuda()
    v = normal((1, H, D), 2).cuda()
    bad = k.clone()
    bad[0, 1, 5] = float("nan")
    worse = v.clone()
    worse[0, 0, 63] = float("-inf")

    def put(n, kk=k, vv=v):
        mx.cache_append(kk, vv, cache, table, i32([n]))
    put(1)
    put(2, bad, worse)
    assert cache.k_scale[2].tolist()[1] == 255 and cache.v_scale[2].tolist()[0] == 255
    assert cache.k_scale[2, 0] != 255 and cache.v_scale[2, 1] != 255
    assert not cache.k[2, 1].any() and not cache.v[2, 0].any() and cache.k[2, 0, :2].any()
    put(3)
    assert cache.k_scale[2, 1] == 255 and not cache.k[2, 1].any()          # stays out
    put(17)
    assert cache.k_scale[1, 1] != 255 and cache.k[1, 1].any()              # the next page is not concerned
    put(1)
    assert cache.k_scale[2, 1] != 255 and cache.k[2, 1, 0].any()           # begun anew


def test_scale_grows_token_by_token():
    """One token at a time with growing values: the codes equal the definition's at every step."""
    page, H, D = 32, 2, 128
    codes, byte, cache, table, _ = setup([page], [0], H, D, page, 3)
    for n in range(1, page + 1):
        k, v = normal((1, H, D), n, 2.0) * 2.0 ** (n // 3), normal((1, H, D), 100 + n, 2.0)
        mx.cache_append(k.cuda(), v.cuda(), cache, i32(table), i32([n]))
        for i, x in enumerate((k, v)):
            codes[i], byte[i] = plain.append((codes[i], byte[i]), x.double().numpy(), table, np.array([n]), np.array([0, 1]))
            assert np.array_equal(to_np(cache[i]), codes[i]) and np.array_equal(to_np(cache[2 + i]), byte[i])


def test_codes_next_to_a_tie_are_the_exact_ones():
    """Rotations whose exact value lies within 2^-30 of a tie between two codes, on either side."""
    H, D, page = 1, 64, 16
    k = torch.zeros((2, H, D), dtype=torch.bfloat16)
    tab = np.zeros((4, D), np.float32)
    tab[:, :32] = 1.0
    # y_0 = x_0 c - x_32 s; 17 (code 16 or 18: a tie) plus or minus less than one fp32 step of it.
    k[:, 0, 0], k[:, 0, 32], k[:, 0, 1] = 17.0, 1.0, 448.0
    tab[0, 32], tab[1, 32] = 2.0 ** -30, -2.0 ** -30
    cache = mx.cache_create(2, H, D, page)
    mx.cache_append(k.cuda(), k.cuda(), cache, i32([[0]]), i32([2]), i32([0, 2]), table=torch.from_numpy(tab).cuda())
    want = plain.append((np.zeros((2, 1, page, D), np.uint8), np.zeros((2, 1), np.uint8)), plain.rope(k.double().numpy(), tab, np.array([0, 1]), False),
                        np.array([[0]]), np.array([2]), np.array([0, 2]))
    assert np.array_equal(to_np(cache.k), want[0]) and np.array_equal(to_np(cache.k_scale), want[1])
    assert plain.decode(want[0])[0, 0, 0, 0] == 16 and plain.decode(want[0])[0, 0, 1, 0] == 18


def test_bad_pages_are_skipped_and_reported():
    H, D, page = 2, 64, 16
    codes, byte, cache, table, _ = setup([40, 40, 40], [1, 1, 1], H, D, page, 4)
    table[1, 2] = 1 << 30
    table[2, 2] = -1
    k, v = normal((3, H, D), 1), normal((3, H, D), 2)
    for offsets in (None, i32([0, 1, 2, 3])):
        mx.device_error()
        mx.cache_append(k.cuda(), v.cuda(), cache, i32(table), i32([40, 40, 70]), offsets)
        assert mx.device_error() == 4
        want = plain.append((codes[0], byte[0]), k.double().numpy(), table, np.array([40, 40, 70]), np.arange(4))
        assert np.array_equal(to_np(cache.k), want[0]) and np.array_equal(to_np(cache.k_scale), want[1])


def test_strided_rows_in_place_queries_and_a_captured_step():
    """k, v and q as views of one fused projection, q rotated in place, the whole call captured and replayed."""
    B, H, Hq, D, page = 5, 2, 6, 128, 16
    lengths = np.array([3, 17, 64, 1, 40])
    codes, byte, cache, table, offsets = setup(lengths, [1] * B, H, D, page, 9)
    tab = plain.table(128, plain.frequencies(D))
    qkv = normal((B, Hq + 2 * H, D), 4).cuda()
    first = qkv.clone()
    args = (cache, i32(table), i32(lengths))
    kw = dict(table=torch.from_numpy(tab).cuda())
    start = [t.clone() for t in cache]
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert mx.cache_append(k, v, *args, q=q, out=q, **kw) is q
    torch.cuda.current_stream().wait_stream(side)
    done = [t.clone() for t in cache]
    want = plain.append((codes[0], byte[0]), plain.rope(first[:, Hq:Hq + H].double().cpu().numpy(), tab, lengths - 1, False), table, lengths, offsets)
    assert np.array_equal(to_np(cache.k), want[0]) and torch.equal(qkv[:, Hq:], first[:, Hq:])
    rotated = qkv.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.cache_append(k, v, *args, q=q, out=q, **kw)
    for t, s in zip(cache, start):
        t.copy_(s)
    qkv.copy_(first)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qkv, rotated) and all(torch.equal(a, b) for a, b in zip(cache, done))
