"""Plain fp64 statements of rotary positions, the paged cache and attention over it (numpy; test infrastructure only).

Nothing here is shared with the library. BF16 tensors come in as float64 arrays of their values."""
import numpy as np

E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])
MID = (E4M3[1:] + E4M3[:-1]) / 2


def encode(x):
    """E4M3 codes of fp64 values: nearest, ties to the even code, beyond the end the largest."""
    a = np.abs(x)
    at = np.searchsorted(MID, a)
    tie = (at < MID.size) & (a == MID[np.minimum(at, MID.size - 1)]) & (at % 2 == 1)
    return ((at + tie) | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def decode(c):
    v = np.append(E4M3, np.nan)[c & 127]
    return np.where(c >= 128, -v, v)


def scale_of(byte):
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def table(positions, freq, amplitude=1.0, first=0):
    a = (first + np.arange(positions))[:, None] * np.asarray(freq)
    return (amplitude * np.concatenate([np.cos(a), np.sin(a)], 1)).astype(np.float32)


def rope(x, tab, pos, interleaved, back=False):
    """x [T, H, D] rotated by rows pos of tab [P, rot]; rows with a position outside the table are zeros."""
    rot = tab.shape[1]
    h = rot // 2
    ok = (pos >= 0) & (pos < tab.shape[0])
    t = tab.astype(np.float64)[np.where(ok, pos, 0)]
    c, s = t[:, None, :h], t[:, None, h:] * (-1 if back else 1)
    y = x.copy()
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(h), np.arange(h, rot))
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    y[~ok] = 0
    return y


def append(cache, x, page_table, lengths, offsets):
    """Codes [P, H, page, D] and scale bytes [P, H] after the rows x [T, H, D] (rotated, fp64) are appended."""
    codes, byte = cache[0].copy(), cache[1].copy()
    page = codes.shape[2]
    for b in range(len(lengths)):
        r0, n = int(offsets[b]), int(offsets[b + 1] - offsets[b])
        start = int(lengths[b]) - n
        first = max(start, 0)
        for p in range(first // page, (int(lengths[b]) - 1) // page + 1 if lengths[b] > first else first // page):
            lo, hi = max(first, p * page), min(int(lengths[b]), (p + 1) * page)
            if p >= page_table.shape[1] or not 0 <= page_table[b, p] < codes.shape[0]:
                continue
            at = page_table[b, p]
            t = x[r0 + lo - start:r0 + hi - start]
            for h in range(codes.shape[1]):
                v = t[:, h]
                old = np.ones(page, bool)          # the page's other codes, where it holds older tokens
                old[lo - p * page:hi - p * page] = False
                old &= lo > p * page
                was = int(byte[at, h]) if lo > p * page else 0
                if not np.isfinite(v).all():
                    s = 255
                else:
                    amax = np.abs(v).max()
                    s = max(int(np.frexp(amax)[1]) - 1 - 8 + 127, 0) if amax > 0 else 0
                s = max(s, was)
                new = slice(lo - p * page, hi - p * page)
                if s == 255:
                    codes[at, h, old] = 0
                    codes[at, h, new] = 0
                else:
                    if s > was:
                        codes[at, h, old] = encode(np.ldexp(decode(codes[at, h, old]), was - s))
                    codes[at, h, new] = encode(np.ldexp(v, 127 - s))
                byte[at, h] = s
    return codes, byte


def attention(q, cache, page_table, lengths, offsets, scale, window=0):
    """(out, lse, sum_j p_j |v_j| / l, largest scale sum_d |q_d k_jd| of a row) of q [T, Hq, D]; NaN rows where a page is bad."""
    k_codes, v_codes, ks, vs = cache
    T, Hq, D = q.shape
    Hkv, page = k_codes.shape[1], k_codes.shape[2]
    G = Hq // Hkv
    out, mass, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    lse = np.full((T, Hq), -np.inf)
    for b in range(len(lengths)):
        r0, n, total = int(offsets[b]), int(offsets[b + 1] - offsets[b]), max(int(lengths[b]), 0)
        pages = -(-total // page)
        if n == 0 or total == 0:
            continue
        ids = np.array([page_table[b, p] if p < page_table.shape[1] else -1 for p in range(pages)])
        ok = (ids >= 0) & (ids < k_codes.shape[0])
        at = np.where(ok, ids, 0)
        for h in range(Hkv):
            def values(codes, byte):
                v = decode(codes[at, h]) * np.where(ok, scale_of(byte[at, h]), np.nan)[:, None, None]
                return v.reshape(-1, D)[:total]
            k, v = values(k_codes, ks), values(v_codes, vs)
            i = total - n + np.arange(n)[:, None]
            j = np.arange(total)[None, :]
            seen = j <= i
            if window > 0:
                seen &= j > i - window
            for g in range(h * G, h * G + G):
                x = q[r0:r0 + n, g]
                with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                    z = np.where(seen, scale * np.einsum("rd,kd->rk", x, k, optimize=True), -np.inf)
                    top = np.where(seen.any(1), z.max(1), 0.0)[:, None]
                    p = np.where(seen, np.exp(z - top), 0.0)
                    l = p.sum(1, keepdims=True)
                    some = seen.any(1)
                    vv = np.where(np.isnan(v), 0.0, v)
                    o = p @ vv
                    poisoned = (seen & np.isnan(v).any(1)[None, :]).any(1)
                    o[poisoned] = np.nan
                    w = p @ np.abs(vv)
                    out[r0:r0 + n, g][some] = (o / l)[some]
                    mass[r0:r0 + n, g][some] = (w / l)[some]
                    lse[r0:r0 + n, g][some] = (top[:, 0] + np.log(l[:, 0]))[some]
                    size[r0:r0 + n, g] = scale * np.where(seen, np.abs(x) @ np.abs(np.nan_to_num(k)).T, 0.0).max(1)
    return out, lse, mass, size
