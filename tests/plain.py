"""Plain fp64 statements of the routing, dispatch, combine and MXFP4 operators (numpy; test infrastructure only).

Nothing here is shared with the library. BF16 tensors come in as float64 arrays of their values."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---- MXFP4 ---------------------------------------------------------------------------------------

def quantize_fp4(x):
    """Rowwise MXFP4 of x [M, K]: (codes uint8 [M, K] with the sign in bit 3, scale bytes uint8 [M, K/32])."""
    M, K = x.shape
    b = np.asarray(x, np.float64).reshape(M, K // 32, 32)
    special = ~np.isfinite(b).all(axis=2)
    a = np.abs(np.where(np.isfinite(b), b, 0.0))
    amax = a.max(axis=2)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)     # floor(log2 amax) - 2
    e = np.clip(e, -127, 127)
    v = np.ldexp(a, -e[:, :, None])
    code = np.zeros(v.shape, np.int64)
    for i in range(7):                                           # past a midpoint, or on one towards the even code
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code += (v > mid) | ((v == mid) & (i % 2 == 1))
    code = np.where(special[:, :, None], 7, code) | (np.signbit(b).astype(np.int64) << 3)
    return code.astype(np.uint8).reshape(M, K), np.where(special, 255, e + 127).astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)


def values_fp4(q, s):
    """fp64 values of packed codes [M, K/2] under raw scale bytes [M, K/32]."""
    code = unpack(q)
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v.reshape(*s.shape, 32) * scale[..., None]).reshape(code.shape)


# ---- routing ---------------------------------------------------------------------------------------

def clean(x):
    """Logits as the operator takes them: NaN as -inf, +inf as the largest finite float."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    return np.minimum(x, np.finfo(np.float32).max)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def scores(x, score):
    """Scores of one row of cleaned logits; experts at -inf score 0."""
    live = x > -np.inf
    if not live.any():
        return np.zeros_like(x)
    if score == "sigmoid":
        return np.where(live, sigmoid(x), 0.0)
    e = np.where(live, np.exp(x - x[live].max()), 0.0)
    return e / e.sum()


def weights_of(x, ids, score, renormalize, scale):
    """The weights of chosen experts ids (those >= 0) of one row, fp64, in the logarithm where sums could underflow."""
    w = np.zeros(len(ids))
    got = np.array([0 <= i < len(x) and x[i] > -np.inf for i in ids], bool)
    if not got.any():
        return w
    z = x[np.asarray(ids)[got]]
    if not renormalize:
        w[got] = scale * scores(x, score)[np.asarray(ids)[got]]
        return w
    log = z if score == "softmax" else np.where(z > 0, -np.log1p(np.exp(-np.abs(z))), z - np.log1p(np.exp(-np.abs(z))))
    r = np.exp(log - log.max())
    w[got] = scale * r / r.sum()
    return w


def route(x, k, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renormalize=True, scale=1.0):
    T, E = x.shape
    x = clean(x)
    ids, weights = np.full((T, k), -1, np.int64), np.zeros((T, k))
    per = E // groups
    for t in range(T):
        by_logit = bias is None and not (groups > topk_groups and group_score == "top2")
        key = x[t].copy() if by_logit else scores(x[t], score)
        if bias is not None:
            key = key + np.asarray(bias, np.float64)
        key = np.where((x[t] > -np.inf) & ~np.isnan(key), key, -np.inf)
        if groups > 1:
            rank = []
            for g in range(groups):
                top = sorted(key[g * per:(g + 1) * per], reverse=True)[:2]
                live = [v for v in top if v > -np.inf]
                rank.append(-np.inf if not live else (live[0] if group_score == "max" else sum(live)))
            order = sorted(range(groups), key=lambda g: (-rank[g], g))[:topk_groups]
            for g in range(groups):
                if g not in order:
                    key[g * per:(g + 1) * per] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:k]
        ids[t, :len(order)] = order
        weights[t] = weights_of(x[t], ids[t], score, renormalize, scale)
    return ids, weights


def route_backward(dw, x, ids, score="softmax", renormalize=True, scale=1.0):
    """(gradient, a magnitude of the terms it sums: what fp32 roundings are relative to)."""
    T, E = x.shape
    x = clean(x)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        got = [j for j, i in enumerate(ids[t]) if 0 <= i < E and x[t, i] > -np.inf]
        if not got:
            continue
        at, g = ids[t, got], np.asarray(dw[t], np.float64)[got]
        p = scores(x[t], score)
        if renormalize:
            r = weights_of(x[t], at, score, True, 1.0)
            c = scale * r * (g - (g * r).sum())
            m = abs(scale) * r * (np.abs(g) + (np.abs(g) * r).sum())
            f = (1.0 - p[at]) if score == "sigmoid" else 1.0
            if score == "sigmoid":
                f = sigmoid(-x[t, at])                       # 1 - s without its cancellation
            np.add.at(d[t], at, c * f)
            np.add.at(size[t], at, m * f)
        elif score == "sigmoid":
            c = scale * g * p[at] * sigmoid(-x[t, at])
            np.add.at(d[t], at, c)
            np.add.at(size[t], at, np.abs(c))
        else:
            c = scale * g * p[at]
            np.add.at(d[t], at, c)
            np.add.at(size[t], at, np.abs(c))
            d[t] -= p * c.sum()
            size[t] += p * np.abs(c).sum()
    return d, size


def plan(ids, E):
    """(row_offsets, slot_row, counts): a stable sort by expert; slots without one last, holding ~row."""
    flat = np.asarray(ids).reshape(-1)
    has = (flat >= 0) & (flat < E)
    key = np.where(has, flat, E)
    order = np.argsort(key, kind="stable")
    row = np.empty(len(flat), np.int64)
    row[order] = np.arange(len(flat))
    counts = np.bincount(key, minlength=E + 1)[:E]
    off = np.concatenate([[0], np.cumsum(counts)])
    off[E] = len(flat)
    return off, np.where(has, row, ~row).reshape(np.asarray(ids).shape), counts


def grouped_layout(raw, off, size):
    """Raw scale bytes [rows, kblocks] as the grouped tensor-core layout of row offsets `off`, zero-filled to `size`."""
    C = (raw.shape[1] + 3) // 4
    out = np.zeros(size, np.uint8)
    tile = 0
    for g in range(len(off) - 1):
        for i, r in enumerate(range(off[g], off[g + 1])):
            for c in range(raw.shape[1]):
                out[((tile + i // 128) * C + c // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + c % 4] = raw[r, c]
        tile += (off[g + 1] - off[g] + 127) // 128
    return out


def combine(rows, slot_row, w):
    """(y, sum of |w c|)."""
    T, k = slot_row.shape
    y, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for j in range(k):
        ok = (slot_row[:, j] >= 0) & (slot_row[:, j] < len(rows))
        term = w[ok, j, None] * rows[slot_row[ok, j]]
        y[ok] += term
        size[ok] += np.abs(term)
    return y, size


def combine_backward(dy, rows, slot_row, w):
    """(d_rows, d_weights, sum of |dy c|); rows that no slot names: NaN."""
    T, k = slot_row.shape
    d_rows, dw, size = np.full(rows.shape, np.nan), np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        s = slot_row[:, j]
        has = s >= 0
        d_rows[np.where(has, s, ~s)] = np.where(has[:, None], w[:, j, None] * dy, 0.0)
        dw[has, j] = (dy[has] * rows[s[has]]).sum(axis=1)
        size[has, j] = np.abs(dy[has] * rows[s[has]]).sum(axis=1)
    return d_rows, dw, size
