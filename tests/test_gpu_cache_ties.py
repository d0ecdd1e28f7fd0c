"""Codes of keys whose rotation lies as near a tie between two codes as BF16 features and fp32 angles allow: those of the exact value.

A feature is x_a c - x_b s. Cases are made so that x_a c misses a tie by a few units 2^-31 of it and x_b s makes up for that but for a few parts
in 2^24 of the miss: what is left is 2^-40 to 2^-56 of the value, on either side, or nothing. Expectations are exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32

pytestmark = pytest.mark.gpu

GRID = [Fraction(float(v)) for v in plain.E4M3]


def code_of(x):
    """E4M3 code of an exact value: the nearest, a tie to the even code."""
    a = abs(x)
    best = min(range(len(GRID)), key=lambda i: (abs(GRID[i] - a), i & 1))
    return best | (128 if x < 0 else 0)


def near_ties(n, seed):
    """(x_a, c, x_b, s) with x_a c - x_b s next to a tie; integers' products, scaled by powers of two at the end."""
    g = np.random.default_rng(seed)
    out = []
    while len(out) < n:
        i = int(g.integers(9, 126))                                     # normal codes but the last
        tie = (GRID[i] + GRID[i + 1]) / 2
        A, B = int(g.integers(64, 128)) * 2 + 1, int(g.integers(64, 128)) * 2 + 1
        # x_a c: the product of A and 24 bits that is nearest the tie; r: what it misses.
        shift = 0
        while tie * 2 ** shift / A < 2 ** 23:
            shift += 1
        C = round(tie * 2 ** shift / A)
        r = A * C - tie * 2 ** shift                                    # in units 2^-shift
        if C >= 2 ** 24 or r == 0:
            continue
        up = 0
        while abs(r) * 2 ** up / B < 2 ** 23:
            up += 1
        S = round(r * 2 ** up / B) + int(g.integers(-1, 2))
        if abs(S) >= 2 ** 24:
            continue
        # Everything in its place: x_a about 1 to 2, c what is left; both signs.
        sign = int(g.choice([-1, 1]))
        out.append((sign * A / 2.0 ** 7, C / 2.0 ** (shift - 7), sign * B / 2.0 ** 7, S / 2.0 ** (shift + up - 7)))
    return out


def check(cases, interleaved, single):
    """A token per case, its own row of the table; the pair's other features: one of 448 that settles the scale, and zeros."""
    D, page, n = 64, 16, len(cases)
    a, b, one = (0, 1, 2) if interleaved else (0, 32, 1)
    k = torch.zeros((n, 1, D), dtype=torch.float64)
    tab = np.zeros((n, D), np.float32)
    tab[:, :32] = 1.0
    for t, (xa, c, xb, s) in enumerate(cases):
        k[t, 0, a], k[t, 0, b], k[t, 0, one] = xa, xb, 448.0
        tab[t, 0], tab[t, 32] = c, s
        assert float(tab[t, 0]) == c and float(tab[t, 32]) == s         # exact in fp32, and in BF16 below
    kb = k.to(torch.bfloat16)
    assert torch.equal(kb.double(), k)
    pages = -(-n // page)
    cache = mx.cache_create(pages, 1, D, page)
    tab_d, zero = torch.from_numpy(tab).cuda(), torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    if single:                                                          # a sequence per case, at the case's position
        table = i32(np.broadcast_to(np.arange(pages), (n, pages)))
        for slot in range(page):                                        # no page twice in a call
            at = np.arange(slot, n, page)
            mx.cache_append(kb[at].cuda(), zero[:len(at)], cache, table[:len(at)], i32(at + 1), table=tab_d, interleaved=interleaved)
    else:
        mx.cache_append(kb.cuda(), zero, cache, i32(np.arange(pages)[None]), i32([n]), i32([0, n]), table=tab_d, interleaved=interleaved)
    assert mx.device_error() == 0
    got, byte = to_np(cache.k).reshape(pages, page, D), to_np(cache.k_scale)[:, 0]
    for p in range(pages):
        want, e = [], -127                                              # codes of features a and b; the page's exponent
        tokens = [tuple(map(Fraction, map(float, case))) for case in cases[p * page:(p + 1) * page]]
        exact = [(xa * c - xb * s, xb * c + xa * s) for xa, c, xb, s in tokens]
        for part in [[y] for y in exact] if single else [exact]:
            grown = max(e, max(int(np.floor(np.log2(float(max(abs(y[0]), abs(y[1]), 448))))) for y in part) - 8)
            want = [tuple(int(plain.encode(np.ldexp(plain.decode(np.uint8(x)), e - grown))) for x in y) for y in want] if grown > e else want
            e = grown
            want += [tuple(code_of(x / Fraction(2) ** e) for x in y) for y in part]
        assert byte[p] == e + 127
        assert [(int(t[a]), int(t[b])) for t in got[p][:len(want)]] == want, p


@pytest.mark.parametrize("single", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_near_ties(interleaved, single):
    check(near_ties(600, 1 + interleaved), interleaved, single)


def test_below_and_above_one_tie():
    """2^-49 below 19/8, a tie whose even code lies above, and as much above and below its negative and 17/8, whose even code lies below."""
    c, s = 13281963 * 2.0 ** -24, 11184811 * 2.0 ** -49
    near = [(3.0, c, 3.0, s), (-3.0, c, -3.0, s), (3.0, c, 3.0, np.nextafter(np.float32(s), np.float32(0)).item()),
            (3.0, 11883862 * 2.0 ** -24, 3.0, -s), (3.0, 11883862 * 2.0 ** -24, 3.0, -np.nextafter(np.float32(s), np.float32(1)).item())]
    for interleaved in (False, True):
        for single in (False, True):
            check(near, interleaved, single)


@pytest.mark.parametrize("power", [-60, -94, -110, -124, -128])
def test_tiny_products(power):
    """Keys so small that the products' last bits, or the products, lie below fp32's subnormals: exact all the same."""
    D, page, n = 64, 16, 400
    g = np.random.default_rng(-power)
    k = torch.from_numpy(np.ldexp(g.integers(-255, 256, (n, 1, D)).astype(np.float64), power - 7)).to(torch.bfloat16)
    tab = (g.integers(1, 1 << 24, (n, D)) * 2.0 ** -24 * np.ldexp(1.0, -g.integers(0, 25, (n, D)))).astype(np.float32)
    cache = mx.cache_create(n // page, 1, D, page)
    mx.cache_append(k.cuda(), k.cuda(), cache, i32(np.arange(n // page)[None]), i32([n]), i32([0, n]), table=torch.from_numpy(tab).cuda())
    byte = to_np(cache.k_scale)[:, 0]
    x, t = k[:, 0].double().numpy(), tab.astype(np.float64)
    got = to_np(cache.k).reshape(n, D)
    y = np.concatenate([x[:, :32] * t[:, :32] - x[:, 32:] * t[:, 32:], x[:, 32:] * t[:, :32] + x[:, :32] * t[:, 32:]], 1)
    want_byte = [max(int(np.frexp(m)[1]) - 9 + 127, 0) for m in np.abs(y).reshape(n // page, -1).max(1)]
    assert np.array_equal(byte, want_byte)
    for i in range(n):
        # fp64's sum decides where it is no tie itself; where it is, exact arithmetic.
        v = np.ldexp(y[i], 127 - int(byte[i // page]))
        want = plain.encode(v)
        for d in np.flatnonzero(np.isin(np.abs(v), plain.MID)):
            h = d % 32
            p, q = Fraction(x[i, d]) * Fraction(t[i, h]), Fraction(x[i, (d + 32) % 64]) * Fraction(t[i, 32 + h])
            want[d] = code_of((p - q if d < 32 else p + q) * Fraction(2) ** (127 - int(byte[i // page])))
        tiny = (y[i] != 0) & (np.abs(y[i]) < 2.0 ** -149)               # 0 of either sign
        assert np.array_equal(got[i] & np.where(tiny, 127, 255), want & np.where(tiny, 127, 255)), i
