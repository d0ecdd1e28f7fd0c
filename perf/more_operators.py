"""Cases for measuring what stands between the qkv and the output projection of a sampler's layer, against plain forms.

Three operators, and one step that runs them together:

  rope    rotary positions of queries and keys (halves or neighbours paired, all or part of the head, scaled tables),
          and the gradient;
  append  new keys and values into a paged cache of E4M3 codes with one E8M0 scale per page and head, the keys and the
          queries rotated on the way;
  attend  attention over that cache: grouped heads, causal against each sequence's end, an optional window, ragged
          batches of prompts and single tokens;
  step    append and attend as a decoding step runs them.

With ``own`` false ``run`` computes them with elementary torch operations in fp32 (fp64 where a code hangs on the last
bits), with ``own`` true through this package. ``exact`` states the definitions once more in fp64.
"""
import math
import random

import torch

own = False

MOST_ROPE = 12288 * 40 * 128          # elements of the largest rotated tensor
MOST_APPEND = 10300 * 8 * 128         # elements of the largest appended key tensor
MOST_CACHE = 4 * 120000 * 4 * 128     # elements of the largest key cache that one pass reads
MOST_PAIRS = 32 * 2048 * 15000        # query heads x rows x keys of the largest score matrix (padded)
TABLE = 131072                        # positions in the rotation tables


# ---- cases ----------------------------------------------------------------------------------------------------------
# attend, append and step: B sequences; `rows` new tokens of the longest one (the others have a quarter to all of it), the last
# `decoding` of them have one new token; `context` tokens of the longest one before the new ones. `mix` draws the lengths.

def listed():
    return [
        # Queries of a decoding step of 13 sequences, far into their contexts.
        dict(name="rope_decode", op="rope", T=13, H=32, D=128, rot=128, interleaved=False, dtype="bf16", scaling="none",
             strided=False, train=False),
        # The 32 query and 8 key heads of a dense update micro-batch (12 288 tokens), inside the qkv projection's
        # 48-head rows, forward and backward.
        dict(name="rope_update", op="rope", T=12288, H=40, D=128, rot=128, interleaved=False, dtype="bf16",
             scaling="none", strided=True, train=True),
        # Half of every head rotated, neighbours paired, positions stretched for long contexts, fp32, an odd batch.
        dict(name="rope_part", op="rope", T=5201, H=12, D=128, rot=64, interleaved=True, dtype="fp32", scaling="yarn",
             strided=False, train=True),
        # One token for each of 64 sequences: keys and values into the cache, queries rotated in the same call.
        dict(name="append_decode", op="append", B=64, rows=1, decoding=64, context=4000, mix=1, Hq=32, Hkv=8, D=128,
             rot=128, page=64, interleaved=False),
        # Five prompts of a rollout, 10 000 tokens in all, some of them behind a cached prefix that ends inside a page.
        dict(name="append_prompt", op="append", B=5, rows=2600, decoding=0, context=300, mix=2, Hq=32, Hkv=8, D=128,
             rot=128, page=64, interleaved=False),
        # A single conversation of a thousand tokens: latency.
        dict(name="attend_one", op="attend", B=1, rows=1, decoding=1, context=1000, mix=3, Hq=32, Hkv=8, D=128, page=64,
             window=0),
        # A sampler's decoding step: 64 sequences of 2000 to 8000 tokens.
        dict(name="attend_decode", op="attend", B=64, rows=1, decoding=64, context=8000, mix=4, Hq=32, Hkv=8, D=128,
             page=64, window=0),
        # Four very long contexts, eight query heads on each key head (the MoE model's heads).
        dict(name="attend_long", op="attend", B=4, rows=1, decoding=4, context=120000, mix=5, Hq=32, Hkv=4, D=128,
             page=128, window=0),
        # Prompts of a rollout: ragged, causal, nothing cached before.
        dict(name="attend_prompt", op="attend", B=6, rows=2048, decoding=0, context=0, mix=6, Hq=32, Hkv=8, D=128,
             page=64, window=0),
        # A piece of a long prompt against the 14 000 tokens in front of it.
        dict(name="attend_chunk", op="attend", B=1, rows=2048, decoding=0, context=14000, mix=7, Hq=32, Hkv=8, D=128,
             page=32, window=0),
        # A sliding window, short heads, small pages: prompts and decoding sequences in one batch.
        dict(name="attend_mixed", op="attend", B=10, rows=700, decoding=7, context=2500, mix=8, Hq=24, Hkv=4, D=64,
             page=16, window=1024),
        # The decoding step whole: 16 sequences, keys and values appended, then attended.
        dict(name="step", op="step", B=16, rows=1, decoding=16, context=3000, mix=9, Hq=32, Hkv=8, D=128, rot=128,
             page=64, interleaved=False, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "step"])
    if op == "rope":
        H, D = _log(rng, 1, 64), rng.choice([64, 80, 96, 128, 192, 256])
        rot = D if rng.random() < 0.5 else rng.choice([16, 32, D // 2 // 2 * 2])
        return dict(op=op, T=min(_log(rng, 1, 20480), MOST_ROPE // (H * D)), H=H, D=D, rot=rot,
                    interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), strided=rng.random() < 0.4, train=rng.random() < 0.5)
    Hkv, D, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    Hq = Hkv * group
    mix = rng.randrange(1 << 20)
    if op == "append":
        B = _log(rng, 1, 128)
        single = rng.random() < 0.4
        rows = 1 if single else max(1, min(_log(rng, 1, 4096), MOST_APPEND // (B * Hkv * D)))
        return dict(op=op, B=B, rows=rows, decoding=B if single else rng.randint(0, B // 2),
                    context=rng.choice([0, _log(rng, 1, 8000)]), mix=mix, Hq=Hq, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2]), page=page, interleaved=rng.random() < 0.4)
    if op == "step":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, rows=1, decoding=B, context=_log(rng, 1, 8000), mix=mix, Hq=Hq, Hkv=Hkv, D=D, rot=D,
                    page=page, interleaved=rng.random() < 0.4, window=0)
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    if rng.random() < 0.5:
        B = _log(rng, 1, 128)
        context = max(1, min(_log(rng, 16, 120000), MOST_CACHE // (B * Hkv * D)))
        return dict(op=op, B=B, rows=1, decoding=B, context=context, mix=mix, Hq=Hq, Hkv=Hkv, D=D, page=page, window=window)
    B, rows = _log(rng, 1, 16), _log(rng, 2, 2048)
    context = rng.choice([0, _log(rng, 16, 14000)])
    rows = max(2, min(rows, MOST_PAIRS // (B * Hq * (context + rows))))
    context = min(context, max(0, MOST_PAIRS // (B * Hq * rows) - rows))
    return dict(op=op, B=B, rows=rows, decoding=rng.randint(0, B - 1), context=context, mix=mix, Hq=Hq, Hkv=Hkv, D=D,
                page=page, window=window)


DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _lengths(c):
    """(new tokens, tokens before them) of every sequence."""
    r = random.Random(c["mix"])
    B, first_single = c["B"], c["B"] - c["decoding"]
    new = [1 if b >= first_single else c["rows"] if b == 0 else r.randint((c["rows"] + 3) // 4, c["rows"]) for b in range(B)]
    before = [c["context"] if b == 0 else r.randint(c["context"] // 4, c["context"]) for b in range(B)]
    return new, before


def _pairs(c):
    """(row, key) pairs of one head that the mask keeps, and keys that any row of a sequence sees."""
    pairs = keys = 0
    for n, a in zip(*_lengths(c)):
        w = c["window"] or a + n
        full = max(0, min(n, w - a))           # rows whose keys all lie in the window
        pairs += full * a + full * (full + 1) // 2 + (n - full) * w
        keys += min(a + n, n + w - 1)
    return pairs, keys


def work(c):
    if c["op"] == "rope":
        esz = 4 if c["dtype"] == "fp32" else 2
        n = c["T"] * c["H"] * c["D"]
        ways = 2 if c["train"] else 1
        return {"bytes": ways * (2 * n * esz + c["T"] * (4 * c["rot"] + 4)), "flops": ways * 3 * c["T"] * c["H"] * c["rot"]}
    T = sum(_lengths(c)[0])
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    b = f = 0
    if c["op"] in ("append", "step"):
        b += T * (2 * Hkv * D * 3 + 2 * Hq * D * 2 + 4 * c["rot"])
        f += T * (3 * (Hq + Hkv) * c["rot"] + 2 * 2 * Hkv * D)
    if c["op"] in ("attend", "step"):
        pairs, keys = _pairs(c)
        b += 2 * keys * Hkv * D + 2 * (keys // c["page"] + c["B"]) * Hkv + T * Hq * D * 4
        f += 4 * pairs * Hq * D
    return {"bytes": b, "flops": f}


# ---- what a program has in hand ---------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _frequencies(rot, scaling):
    """(angle per position of every pair, factor on cosine and sine), in fp64."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 1e6 ** (-2 * i / rot)
    if scaling == "linear":
        return f / 4, 1.0
    if scaling == "yarn":          # stretched 4 times beyond 32 768 positions: slow pairs by the factor, fast ones not at all
        at = [rot * math.log(32768 / (2 * math.pi * turns)) / (2 * math.log(1e6)) for turns in (32, 1)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / 4 * ramp + f * (1 - ramp), 0.1 * math.log(4) + 1
    return f, 1.0


def _table(rot, scaling="none", positions=TABLE):
    """fp32 [positions, rot]: the cosines of a position's angles, then the sines."""
    f, m = _frequencies(rot, scaling)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return (m * torch.cat([torch.cos(a), torch.sin(a)], dim=1)).float()


def _keys(g, *shape):
    """Keys and values as projections give them: N(0, 1) under a lognormal scale per channel."""
    return _randn(g, *shape) * torch.exp(0.5 * _randn(g, shape[-3] if len(shape) == 4 else 1, 1, shape[-1]))


def _codes(x):
    """E4M3 codes and scale bytes [P, H] of pages [P, H, page, D] in fp32."""
    e = _exponent(x.abs().amax(dim=(2, 3)))
    return _e4m3(x * _pow2(-e)[:, :, None, None]).view(torch.uint8), (e + 127).to(torch.uint8)


def _batch(c, g, s):
    """Lengths, row offsets, a page table over shuffled pages (entries behind a sequence's end: page 0) and the cache."""
    new, before = _lengths(c)
    total = [a + n for n, a in zip(new, before)]
    need = [-(-t // c["page"]) for t in total]
    width = max(need) + 1
    s["T"], s["most"], s["longest"] = sum(new), max(new), max(total)
    pages = sum(need) + 7
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")[None, :]
    have = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(have, 0) - have
    s["page_table"] = torch.where(col < have, order[(first + col).clamp(max=pages - 1)], torch.zeros_like(order[:1])).contiguous()
    s["lengths"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    s["row_offsets"] = None if max(new) == 1 else torch.tensor(off, dtype=torch.int32, device="cuda")
    shape = (pages, c["Hkv"], c["page"], c["D"])
    k, ks = _codes(_keys(g, *shape))
    v, vs = _codes(_keys(g, *shape))
    s["cache"] = (k, v, ks, vs)


def prepare(c, seed):
    g, op = _gen(seed), c["op"]
    s = {"c": c}
    if op == "rope":
        T, H, D, dt = c["T"], c["H"], c["D"], DTYPES[c["dtype"]]
        wide = H + 8 if c["strided"] else H
        s["x"] = _randn(g, T, wide, D).to(dt)[:, :H]
        s["dy"] = _randn(g, T, H, D).to(dt) if c["train"] else None
        s["table"] = _table(c["rot"], c["scaling"])
        start = torch.randint(0, TABLE - T, (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        return s
    _batch(c, g, s)
    T, Hq, Hkv, D = s["T"], c["Hq"], c["Hkv"], c["D"]
    s["q"] = _randn(g, T, Hq, D).to(torch.bfloat16)
    if op != "attend":
        s["table"] = _table(c["rot"])
        s["k"] = _keys(g, T, Hkv, D).to(torch.bfloat16)
        s["v"] = _keys(g, T, Hkv, D).to(torch.bfloat16)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------

def _exponent(amax):
    """floor(log2 amax) - 8, at least -127 (also for 0)."""
    e = torch.frexp(amax).exponent - 9
    return torch.where(amax > 0, e.clamp(min=-127), torch.full_like(e, -127))


def _pow2(e, dtype=torch.float32):
    return torch.ldexp(torch.ones((), dtype=dtype, device=e.device), e)


def _e4m3(x):
    """Nearest E4M3 value, ties to even, at most 448, in the arithmetic of x."""
    step = _pow2((torch.frexp(x.abs().clamp(min=2.0 ** -20)).exponent - 1).clamp(min=-6) - 3, x.dtype)
    return (torch.round(x / step) * step).clamp(-448, 448).float().to(torch.float8_e4m3fn)


def _rotated(x, cos, sin, rot, interleaved):
    """x [T, H, D] with cos and sin [T, rot / 2], in the arithmetic of x."""
    cos, sin = cos[:, None, :].to(x.dtype), sin[:, None, :].to(x.dtype)
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], dim=-1).flatten(-2) if interleaved else torch.cat([ya, yb], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _rows(s):
    """(sequence, place among the sequence's new tokens, position) of every row."""
    n = torch.ones_like(s["lengths"]) if s["row_offsets"] is None else s["row_offsets"].diff()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n.long(), output_size=s["T"])
    place = torch.arange(s["T"], device="cuda") - (torch.cumsum(n, 0) - n)[seq]
    return seq, place, (s["lengths"] - n)[seq] + place


def _append(s):
    c, (ck, cv, ks, vs) = s["c"], s["cache"]
    rot, page = c["rot"], c["page"]
    seq, _, pos = _rows(s)
    at, slot = s["page_table"][seq, pos // page].long(), pos % page
    cos, sin = s["table"][pos, :rot // 2], s["table"][pos, rot // 2:]
    touched = torch.zeros(ck.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, at, True)
    fresh = torch.zeros_like(touched).index_fill_(0, at[slot == 0], True)
    kept = (touched & ~fresh)[:, None]
    some = torch.nonzero(touched).reshape(-1)
    # Codes hang on the last bits of the rotation: fp64.
    for x, code, byte in ((_rotated(s["k"].double(), cos, sin, rot, c["interleaved"]), ck, ks), (s["v"].double(), cv, vs)):
        amax = torch.zeros(byte.shape, dtype=torch.float64, device="cuda")
        amax.scatter_reduce_(0, at[:, None].expand(-1, c["Hkv"]), x.abs().amax(dim=2), "amax")
        was = byte.int() - 127
        e = torch.where(kept, torch.maximum(was, _exponent(amax)), _exponent(amax))
        e = torch.where(touched[:, None], e, was)
        old = code[some].view(torch.float8_e4m3fn).float() * _pow2((was - e)[some])[:, :, None, None]
        code[some] = torch.where((kept & (e > was))[some][:, :, None, None], _e4m3(old).view(torch.uint8), code[some])
        code[at, :, slot] = _e4m3(x * _pow2(-e, torch.float64)[at][:, :, None]).view(torch.uint8)
        byte.copy_((e + 127).to(torch.uint8))
    return _rotated(s["q"].float(), cos, sin, rot, c["interleaved"]).to(torch.bfloat16)


def _attend(s, q):
    c, (ck, cv, ks, vs) = s["c"], s["cache"]
    B, Hq, Hkv, D, page, n = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], s["most"]
    seq, place, pos = _rows(s)
    pages = s["page_table"][:, :-(-s["longest"] // page)].long()

    def values(code, byte):
        x = code[pages].view(torch.float8_e4m3fn).float() * _pow2(byte[pages].int() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)

    k, v = values(ck, ks), values(cv, vs)
    qp = torch.zeros((B, n, Hq, D), dtype=torch.float32, device="cuda")
    qp[seq, place] = q.float()
    qp = qp.view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(qp, k.transpose(2, 3)) * D ** -0.5
    last = torch.full((B, n), -1, dtype=torch.int64, device="cuda")
    last[seq, place] = pos.long()
    key = torch.arange(k.shape[2], device="cuda")
    seen = key <= last[:, :, None]
    if c["window"]:
        seen &= key > last[:, :, None] - c["window"]
    score = score.view(B, Hkv, Hq // Hkv, n, -1)
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(dim=-1, keepdim=True).clamp_(min=-1e30)
    p = score.sub_(top).exp_()
    z = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, -1, k.shape[2]), v).view(B, Hkv, Hq // Hkv, n, D)
    out = out / torch.where(z > 0, z, torch.ones_like(z))
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[seq, place].to(torch.bfloat16)


def _whole_cache(s):
    k, v, ks, vs = s["cache"]
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn),
            "k_scale": ks.view(torch.float8_e8m0fnu), "v_scale": vs.view(torch.float8_e8m0fnu)}


def _plain(s):
    c = s["c"]
    if c["op"] == "rope":
        rot, table = c["rot"], s["table"][s["positions"]]
        cos, sin = table[:, :rot // 2], table[:, rot // 2:]
        out = {"y": _rotated(s["x"].float(), cos, sin, rot, c["interleaved"]).to(s["x"].dtype)}
        if c["train"]:
            out["dx"] = _rotated(s["dy"].float(), cos, -sin, rot, c["interleaved"]).to(s["x"].dtype)
        return out
    if c["op"] == "attend":
        return _attend(s, s["q"])
    q = _append(s)
    return {"q": q, **_whole_cache(s)} if c["op"] == "append" else {"out": _attend(s, q), **_whole_cache(s)}


def run(s):
    if not own:
        return _plain(s)
    from mxfp8_block_scaled_07_b200 import mx

    c = s["c"]
    if c["op"] == "rope":
        out = {"y": mx.rope(s["x"], s["table"], s["positions"], interleaved=c["interleaved"])}
        if c["train"]:
            out["dx"] = mx.rope_backward(s["dy"], s["table"], s["positions"], interleaved=c["interleaved"])
        return out
    where = (s["cache"], s["page_table"], s["lengths"], s["row_offsets"])
    if c["op"] == "attend":
        return mx.cache_attention(s["q"], *where, window=c["window"])
    q = mx.cache_append(s["k"], s["v"], *where, q=s["q"], table=s["table"], interleaved=c["interleaved"])
    if c["op"] == "append":
        return {"q": q, **_whole_cache(s)}
    return {"out": mx.cache_attention(q, *where), **_whole_cache(s)}


# ---- definitions in fp64 -----------------------------------------------------------------------------------------------

E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(x):
    """Every fp64 value's nearest E4M3 value, ties to the even code, beyond the end to the largest."""
    grid = torch.tensor(E4M3, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    at = torch.searchsorted(mid, a.contiguous())
    tie = (at < mid.numel()) & (a == mid[at.clamp(max=mid.numel() - 1)]) & (at % 2 == 1)
    return torch.copysign(grid[at + tie.long()], x)


def _turned(x, table, interleaved, back=False):
    """x [T, H, D] times the rotations of table rows [T, rot], as complex numbers in fp64."""
    t = table.double()
    h = t.shape[1] // 2
    turn = torch.complex(t[:, :h], -t[:, h:] if back else t[:, h:])[:, None, :]
    y = x.double().clone()
    part = y[..., :2 * h]
    pair = part.unflatten(-1, (h, 2)) if interleaved else part.unflatten(-1, (2, h)).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * turn
    pair.copy_(torch.view_as_real(z))
    return y


def _cache64(cache):
    k, v, ks, vs = cache
    decode = torch.cat([torch.tensor(E4M3, dtype=torch.float64), torch.tensor([float("nan")], dtype=torch.float64)]).cuda()
    decode = torch.cat([decode, -decode])
    power = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [float("nan")], dtype=torch.float64, device="cuda")
    return decode, power


def _append64(c, s):
    """The cache's codes (as values) and scales after the call, page by page of every sequence."""
    codes, power = _cache64(s["cache"])
    new, before = _lengths(c)
    out = {}
    row = 0
    rows = []
    for n in new:
        rows.append((row, row + n))
        row += n
    pos = torch.cat([torch.arange(a, a + n, device="cuda") for n, a in zip(new, before)])
    inputs = {"k": _turned(s["k"], s["table"][pos], c["interleaved"]), "v": s["v"].double()}
    for name, code, byte in (("k", s["cache"][0], s["cache"][2]), ("v", s["cache"][1], s["cache"][3])):
        value, scale = codes[code.long()], power[byte.long()]
        x = inputs[name]
        for b, (n, a) in enumerate(zip(new, before)):
            for p in range(a // c["page"], (a + n - 1) // c["page"] + 1):
                lo, hi = max(a, p * c["page"]), min(a + n, (p + 1) * c["page"])
                t = x[rows[b][0] + lo - a:rows[b][0] + hi - a].transpose(0, 1)          # [H, tokens, D]
                at = int(s["page_table_host"][b][p])
                # The largest power of two that is at most amax, over 2^8.
                sc = power[(torch.searchsorted(power[:255], t.abs().amax(dim=(1, 2)), right=True) - 9).clamp(min=0)]
                if lo > p * c["page"]:
                    sc = torch.maximum(sc, scale[at])
                    value[at] = torch.where((sc > scale[at])[:, None, None], _nearest(value[at] * (scale[at] / sc)[:, None, None]), value[at])
                value[at, :, lo - p * c["page"]:hi - p * c["page"]] = _nearest(t / sc[:, None, None])
                scale[at] = sc
        out[name], out[name + "_scale"] = value, scale
    return out


def _attend64(c, s, q, values, scales):
    """values: codes of k and v, or what they stand for; scales likewise. One sequence and one key head at a time."""
    codes = _cache64(s["cache"])[0]
    new, before = _lengths(c)
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, a) in enumerate(zip(new, before)):
        pages = s["page_table"][b, :-(-(a + n) // c["page"])].long()
        i = torch.arange(a, a + n, device="cuda")[:, None]
        j = torch.arange(a + n, device="cuda")[None, :]
        out_of_sight = (j > i) | (j <= i - c["window"] if c["window"] else j < 0)
        for h in range(c["Hkv"]):
            k, v = (x[pages, h] for x in values)
            k, v = (codes[x.long()] if x.dtype == torch.uint8 else x for x in (k, v))
            k, v = ((x * sc[pages, h][:, None, None]).reshape(-1, c["D"])[:a + n] for x, sc in zip((k, v), scales))
            for g in range(G):
                z = torch.einsum("rd,kd->rk", q[row:row + n, h * G + g].double(), k) / math.sqrt(c["D"])
                z[out_of_sight] = float("-inf")
                out[row:row + n, h * G + g] = torch.einsum("rk,kd->rd", torch.softmax(z, dim=1), v)
        row += n
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        t = s["table"][s["positions"]]
        out = {"y": _turned(s["x"], t, c["interleaved"])}
        if c["train"]:
            out["dx"] = _turned(s["dy"], t, c["interleaved"], back=True)
        return out
    if c["op"] == "attend":
        power = _cache64(s["cache"])[1]
        k, v, ks, vs = s["cache"]
        return _attend64(c, s, s["q"], [k, v], [power[ks.long()], power[vs.long()]])
    s["page_table_host"] = s["page_table"].tolist()
    new, before = _lengths(c)
    pos = torch.cat([torch.arange(a, a + n, device="cuda") for n, a in zip(new, before)])
    q = _turned(s["q"], s["table"][pos], c["interleaved"])
    made = _append64(c, s)
    if c["op"] == "append":
        return {"q": q, **made}
    out = _attend64(c, s, q.to(torch.bfloat16), [made["k"], made["v"]], [made["k_scale"], made["v_scale"]])
    return {"out": out, **made}
