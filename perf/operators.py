"""Cases for measuring the routed-expert and 4-bit operators against their plain forms.

Five operators, each with a forward form and, where a learner trains through it, its backward:

  route     router logits [T, E] -> the k experts of every token and their weights, and the gradient of the logits;
  dispatch  the experts' row partition of a batch, and the tokens quantized to MXFP8 into the experts' rows;
  combine   the experts' rows weighted and summed back into tokens, and the gradients of rows and weights;
  quantize  BF16 -> MXFP4 (E2M1 codes, one E8M0 scale per 32), rowwise and columnwise, and back to BF16;
  product   block-scaled MXFP4 products, dense and for routed experts.

With ``own`` false ``run`` computes them with elementary torch operations in fp32 (fp64 where a selection hangs on
the last bits), with ``own`` true through this package. ``exact`` states the definitions once more in fp64.
"""
import torch

own = False

MOST_ROUTE = 20480 * 128           # tokens x experts of the largest router case
MOST_ROWS = 20480 * 8 * 2048       # routed rows x features of the largest dispatch and combine cases
MOST_QUANT = 12288 * 4096          # elements of the largest quantized tensor
MOST_FLOPS = 2 * 5200 * 24576 * 4096


# ---- cases ----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # A decoding step of 16 sequences through a large router: 256 experts in 8 groups, sigmoid scores, balance bias.
        dict(name="route_decode", op="route", T=16, E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             group_score="top2", renorm=True, scale=2.5, dtype="fp32", train=False, masked=False),
        # The router of one MoE update micro-batch (20 480 tokens, top-8 of 128), forward and backward.
        dict(name="route_update", op="route", T=20480, E=128, k=8, score="softmax", bias=False, groups=1,
             topk_groups=1, group_score="max", renorm=True, scale=1.0, dtype="bf16", train=True, masked=False),
        # A ragged prompt batch with switched-off experts and padding tokens: odd sizes, bias under a softmax.
        dict(name="route_ragged", op="route", T=5201, E=100, k=6, score="softmax", bias=True, groups=10, topk_groups=5,
             group_score="max", renorm=False, scale=1.5, dtype="bf16", train=True, masked=True),
        # A decoding step's tokens into the experts' rows; a few of them are padding of the captured batch.
        dict(name="dispatch_decode", op="dispatch", T=13, E=128, k=8, K=2048, dropped=True),
        # The update micro-batch's tokens into 163 840 expert rows.
        dict(name="dispatch_update", op="dispatch", T=20480, E=128, k=8, K=2048, dropped=False),
        # The decoding step's expert outputs back into tokens.
        dict(name="combine_decode", op="combine", T=13, E=128, k=8, N=2048, dropped=True, dtype="bf16", train=False),
        # The update micro-batch's expert outputs, forward and backward.
        dict(name="combine_update", op="combine", T=20480, E=128, k=8, N=2048, dropped=False, dtype="bf16", train=True),
        # A small tensor (256 x 512), where the launch counts.
        dict(name="quantize_small", op="quantize", M=256, K=512, col=False),
        # Activations of a dense update micro-batch: the rowwise copy of fprop and the columnwise copy of wgrad.
        dict(name="quantize_update", op="quantize", M=12288, K=4096, col=True),
        # A sampler's decoding step through the qkv projection: 16 rows, bound by the 4-bit weight's bytes.
        dict(name="product_decode", op="product", M=16, N=6144, K=4096, out="bf16"),
        # The gate_up projection of a 5200-token micro-batch.
        dict(name="product_forward", op="product", M=5200, N=24576, K=4096, out="bf16"),
        # Tokens in hand, quantized to 4 bits into their experts' rows, times the experts' gate_up weights.
        dict(name="product_experts", op="experts", T=2048, E=32, k=4, N=1536, K=2048, dropped=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "combine", "quantize", "product", "experts"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384])
        groups = rng.choice([1, 1] + [g for g in (2, 4, 5, 8) if E % g == 0 and E // g >= 4])
        topk_groups = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(8, topk_groups * (E // groups)))
        return dict(op=op, T=min(_log(rng, 1, 20480), MOST_ROUTE // E), E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.5, 2.5]), dtype=rng.choice(["bf16", "fp32"]), train=rng.random() < 0.5,
                    masked=rng.random() < 0.4)
    if op in ("dispatch", "combine"):
        E, k = rng.choice([8, 16, 60, 64, 128, 256]), rng.randint(1, 8)
        width = 32 * _log(rng, 2, 192)
        T = max(1, min(_log(rng, 1, 20480), MOST_ROWS // (k * width)))
        if op == "dispatch":
            return dict(op=op, T=T, E=E, k=k, K=width, dropped=rng.random() < 0.4)
        return dict(op=op, T=T, E=E, k=k, N=width - rng.choice([0, 0, 1, 8]), dropped=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "fp32"]), train=rng.random() < 0.5)
    if op == "quantize":
        col = rng.random() < 0.5
        K = 32 * _log(rng, 1, 384)
        M = max(1, min(_log(rng, 1, 24576), MOST_QUANT // K))
        return dict(op=op, M=max(32, M // 32 * 32) if col else M, K=K, col=col)
    if op == "product":
        M, N, K = _log(rng, 1, 12288), _log(rng, 40, 24576), 32 * _log(rng, 1, 384)
        M = max(1, min(M, MOST_FLOPS // (2 * N * K)))
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "fp32"]))
    E, k = rng.choice([4, 8, 16, 32]), rng.randint(1, 4)
    return dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, N=_log(rng, 64, 2048), K=32 * _log(rng, 2, 64),
                dropped=rng.random() < 0.4, out=rng.choice(["bf16", "fp32"]))


DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def work(c):
    op = c["op"]
    if op == "route":
        esz = 2 if c["dtype"] == "bf16" else 4
        cells, slots = c["T"] * c["E"], c["T"] * c["k"]
        fwd = cells * esz + slots * 8 + (4 * c["E"] if c["bias"] else 0)
        return {"bytes": fwd + (2 * cells * esz + slots * 8 if c["train"] else 0), "flops": cells * (12 if c["train"] else 4)}
    if op == "dispatch":
        rows = c["T"] * c["k"]
        return {"bytes": rows * 4 + rows * 4 + c["E"] * 8 + c["T"] * c["K"] * 2 + rows * c["K"] * 33 // 32,
                "flops": 2 * c["T"] * c["K"]}
    if op == "combine":
        esz = 2 if c["dtype"] == "bf16" else 4
        rows = c["T"] * c["k"]
        fwd = rows * c["N"] * esz + rows * 8 + c["T"] * c["N"] * esz
        bwd = 2 * rows * c["N"] * esz + rows * 12 + c["T"] * c["N"] * esz
        return {"bytes": fwd + (bwd if c["train"] else 0), "flops": rows * c["N"] * (5 if c["train"] else 2)}
    if op == "quantize":
        n = c["M"] * c["K"]
        ways = 2 if c["col"] else 1
        return {"bytes": 2 * n + ways * (2 * (n // 2 + n // 32) + 2 * n), "flops": 3 * ways * n}
    esz = 2 if c["out"] == "bf16" else 4
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * K * 17 // 32 + M * N * esz, "flops": 2 * M * N * K}
    rows, N, K = c["T"] * c["k"], c["N"], c["K"]
    return {"bytes": rows * 8 + c["T"] * K * 2 + 2 * rows * K * 17 // 32 + min(c["E"], rows) * N * K * 17 // 32 + rows * N * esz,
            "flops": 2 * rows * N * K}


# ---- what a program has in hand ---------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _experts_of(g, T, E, k, dropped):
    """k distinct experts per token, popularity ~ rank^-1.1 as in the repository's routed workload; padding tokens
    (the last eighth, at least one) have none."""
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
    ids = torch.topk(-1.1 * torch.log(rank.float()) - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)
    if dropped:
        ids[T - max(1, T // 8):] = -1
    return ids.contiguous()


def _activations(g, M, K):
    """N(0, 1) with a per-channel lognormal scale, as activations have it."""
    return (_randn(g, M, K) * torch.exp(_randn(g, 1, K))).to(torch.bfloat16)


def prepare(c, seed):
    g, op = _gen(seed), c["op"]
    s = {"c": c}
    if op == "route":
        T, E = c["T"], c["E"]
        x = 1.5 * _randn(g, T, E) + _randn(g, 1, E)
        if c["masked"]:
            off = torch.rand((E,), generator=g, device="cuda") < 0.1
            x[:, off] = float("-inf")
            x[T - max(1, T // 16):] = float("-inf")
        s["logits"] = x.to(DTYPES[c["dtype"]])
        s["bias"] = 0.05 * _randn(g, E) if c["bias"] else None
        s["d_weights"] = _randn(g, T, c["k"]) if c["train"] else None
    elif op == "dispatch":
        s["ids"] = _experts_of(g, c["T"], c["E"], c["k"], c["dropped"])
        s["x"] = _activations(g, c["T"], c["K"])
    elif op == "combine":
        T, k, N, dt = c["T"], c["k"], c["N"], DTYPES[c["dtype"]]
        ids = _experts_of(g, T, c["E"], k, c["dropped"])
        s["slot_row"] = _plan(ids, c["E"])[1]
        w = torch.softmax(_randn(g, T, k), dim=1)
        s["weights"] = torch.where(ids >= 0, w, torch.zeros_like(w))
        s["rows"] = _randn(g, T * k, N).to(dt)
        s["dy"] = _randn(g, T, N).to(dt) if c["train"] else None
    elif op == "quantize":
        s["x"] = _activations(g, c["M"], c["K"])
    elif op == "product":
        for n, x in (("a", _activations(g, c["M"], c["K"])), ("b", 0.02 * _randn(g, c["N"], c["K"]))):
            codes, e = _mxfp4(x.float())
            s["q" + n], s["s" + n] = _pack(codes), _to_layout(_byte(e))
    else:
        s["ids"] = _experts_of(g, c["T"], c["E"], c["k"], c["dropped"])
        s["x"] = _activations(g, c["T"], c["K"])
        codes, e = _mxfp4(0.02 * _randn(g, c["E"], c["N"], c["K"]))
        s["qb"], s["sb"] = _pack(codes), torch.cat([_to_layout(b) for b in _byte(e)])
        key = torch.where(s["ids"] >= 0, s["ids"], c["E"] - 1)
        s["most"] = int(torch.bincount(key.reshape(-1).long(), minlength=c["E"]).max())
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------

def _first_k(keys, k):
    """Indices of the k largest along the last axis, largest first, ties to the lowest index."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :k]


def _scores(x, score):
    if score == "softmax":
        m = x.amax(dim=1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        z = e.sum(dim=1, keepdim=True)
        return e / torch.where(z > 0, z, torch.ones_like(z))
    return torch.where(torch.isinf(x), torch.zeros_like(x), 1 / (1 + torch.exp(-x)))


def _route(x, bias, c):
    """ids, weights and the scores' parts that the backward needs."""
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    dead = torch.isinf(x)
    # The choice: in fp64, since two scores may lie nearer together than fp32 tells apart.
    x64 = x.double()
    key = x64 if bias is None and not (G > 1 and c["group_score"] == "top2") else _scores(x64, c["score"])
    if bias is not None:
        key = key + bias.double()
    key = torch.where(dead, torch.full_like(key, float("-inf")), key)
    if G > 1:
        per = key.view(T, G, E // G)
        if c["group_score"] == "max":
            rank = per.amax(dim=2)
        else:
            top = torch.sort(per, dim=2, descending=True).values[:, :, :2]
            rank = torch.where(torch.isinf(top[:, :, 0]), top[:, :, 0],
                               torch.where(torch.isinf(top), torch.zeros_like(top), top).sum(dim=2))
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        kept.scatter_(1, _first_k(rank, c["topk_groups"]), True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, torch.full_like(key, float("-inf")))
    ids = _first_k(key, k)
    none = torch.isinf(torch.gather(key, 1, ids))
    # The weights: in fp32.
    p = _scores(x.float(), c["score"])
    chosen = torch.where(none, torch.zeros_like(p[:, :1]), torch.gather(p, 1, ids))
    total = chosen.sum(dim=1, keepdim=True) if c["renorm"] else torch.ones_like(chosen[:, :1])
    total = torch.where(total > 0, total, torch.ones_like(total))
    w = c["scale"] * chosen / total
    return torch.where(none, -1, ids).to(torch.int32), w, p, chosen, total, none


def _route_backward(dw, ids, p, chosen, total, none, c):
    dw = torch.where(none, torch.zeros_like(dw), dw)
    r = chosen / total
    d_score = c["scale"] / total * (dw - (dw * r).sum(dim=1, keepdim=True) if c["renorm"] else dw)
    d = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0).long(), torch.where(none, torch.zeros_like(d_score), d_score))
    if c["score"] == "softmax":
        return p * (d - (d * p).sum(dim=1, keepdim=True))
    return d * p * (1 - p)


def _plan(ids, E):
    """(row offsets [E + 1], row of every slot, tokens per expert): slots sorted by expert, in slot order within one;
    slots without an expert come last, as padding rows of the last expert, and hold ~row."""
    flat = ids.reshape(-1)
    has = flat >= 0
    key = torch.where(has, flat, E).long()
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order).scatter_(0, order, torch.arange(key.numel(), device=key.device))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=key.device).scatter_add_(0, key, torch.ones_like(key))
    off = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts[:E], 0)])
    off[E] = key.numel()
    return off.to(torch.int32), torch.where(has, row, ~row).to(torch.int32).view(ids.shape), counts[:E].to(torch.int32)


def _block_exponent(x, emax):
    """floor(log2 amax) - emax of every block of 32 along the last axis, at least -127; an all-zero block gets -127."""
    amax = x.reshape(*x.shape[:-1], -1, 32).abs().amax(dim=-1)
    e = torch.frexp(amax).exponent - 1 - emax
    return torch.where(amax > 0, e.clamp(min=-127), torch.full_like(e, -127))


def _byte(e):
    return (e + 127).to(torch.uint8)


def _pow2(e):
    """2^e in fp32 for -127 <= e <= 127."""
    return torch.where(e > -127, ((e + 127).clamp(min=1) << 23), torch.full_like(e, 1 << 22)).to(torch.int32).view(torch.float32)


def _scaled(x, e):
    return x.reshape(*x.shape[:-1], -1, 32) * _pow2(-e).unsqueeze(-1)


def _mxfp8(x):
    e = _block_exponent(x, 8)
    return _scaled(x, e).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(x.shape), e


def _mxfp4(x):
    """E2M1 codes (sign in bit 3) and block exponents of fp32 values."""
    e = _block_exponent(x, 2)
    v = _scaled(x, e).reshape(x.shape)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6)          # round half to even is E2M1's tie to the even code here
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    return code | (torch.signbit(v).to(torch.uint8) << 3), e


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values4(q):
    """The fp32 values of packed E2M1 codes."""
    code = torch.stack([q & 15, q >> 4], dim=-1).reshape(*q.shape[:-1], -1)
    m = (code & 7).float()
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(code >= 8, -a, a)


def _to_layout(raw, padded_rows=None):
    """The tensor-core scale layout of raw scale bytes [rows, kblocks]."""
    R, C = raw.shape
    full = torch.zeros(((R + 127) // 128 * 128, (C + 3) // 4 * 4), dtype=torch.uint8, device=raw.device)
    full[:R, :C] = raw
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _from_layout(s, R, C):
    ct = (C + 3) // 4
    return s.view(-1, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * ct)[:R, :C]


def _dequantized4(q, raw):
    v = _values4(q)
    return (v.reshape(*v.shape[:-1], -1, 32) * _pow2(raw.int() - 127).unsqueeze(-1)).reshape(v.shape)


def _plain(s):
    c = s["c"]
    op = c["op"]
    if op == "route":
        ids, w, p, chosen, total, none = _route(s["logits"], s["bias"], c)
        if not c["train"]:
            return {"ids": ids, "weights": w}
        d = _route_backward(s["d_weights"], ids, p, chosen, total, none, c)
        return {"ids": ids, "weights": w, "d_logits": d.to(s["logits"].dtype)}
    if op == "dispatch":
        E, kb = c["E"], c["K"] // 32
        off, slot_row, counts = _plan(s["ids"], E)
        codes, e = _mxfp8(s["x"].float())
        slot = slot_row.reshape(-1).long()
        has = slot >= 0
        row = torch.where(has, slot, ~slot)
        token = torch.arange(c["T"], device=row.device).repeat_interleave(c["k"])
        q = torch.zeros((row.numel(), c["K"]), dtype=torch.uint8, device=row.device)
        q[row] = torch.where(has[:, None], codes.view(torch.uint8)[token], torch.zeros_like(q))
        sizes = (off[1:] - off[:-1]).long()
        padded = torch.cumsum((sizes + 127) // 128 * 128, 0)
        first = torch.cat([torch.zeros_like(padded[:1]), padded[:-1]])
        expert = torch.searchsorted(off[1:].contiguous(), row.int(), right=True)
        at = first[expert] + row - off[:-1].long()[expert]
        raw = torch.zeros(((row.numel() + 127 * min(E, row.numel())) // 128 * 128, kb), dtype=torch.uint8, device=row.device)
        raw[at] = torch.where(has[:, None], _byte(e)[token], torch.zeros_like(raw[:1]))
        return {"offsets": off, "slot_row": slot_row, "counts": counts, "codes": q.view(torch.float8_e4m3fn),
                "scales": _to_layout(raw).view(torch.float8_e8m0fnu)}
    if op == "combine":
        slot, w, rows = s["slot_row"].long(), s["weights"], s["rows"]
        has = slot >= 0
        picked = rows[slot.clamp(min=0)].float()                                    # [T, k, N]
        y = (torch.where(has, w, torch.zeros_like(w)).unsqueeze(-1) * picked).sum(dim=1).to(rows.dtype)
        if not c["train"]:
            return {"y": y}
        dy = s["dy"].float()
        dw = torch.where(has, (picked * dy.unsqueeze(1)).sum(dim=2), torch.zeros_like(w))
        d_rows = torch.empty_like(rows)
        d_rows[torch.where(has, slot, ~slot).reshape(-1)] = (
            torch.where(has, w, torch.zeros_like(w)).unsqueeze(-1) * dy.unsqueeze(1)).to(rows.dtype).reshape(rows.shape)
        return {"y": y, "d_rows": d_rows, "d_weights": dw}
    if op == "quantize":
        out = {}
        for way in ("row", "col") if c["col"] else ("row",):
            x = s["x"].float() if way == "row" else s["x"].float().t().contiguous()
            codes, e = _mxfp4(x)
            q = _pack(codes)
            out["scales_" + way] = _to_layout(_byte(e)).view(torch.float8_e8m0fnu)
            out["values_" + way] = _dequantized4(q, _byte(e)).to(torch.bfloat16)
        return out
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        a = _dequantized4(s["qa"], _from_layout(s["sa"], M, K // 32))
        b = _dequantized4(s["qb"], _from_layout(s["sb"], N, K // 32))
        return (a @ b.t()).to(DTYPES[c["out"]])
    E, N, K = c["E"], c["N"], c["K"]
    off, slot_row, _ = _plan(s["ids"], E)
    codes, e = _mxfp4(s["x"].float())
    xq = _dequantized4(_pack(codes), _byte(e))
    slot = slot_row.reshape(-1).long()
    row = torch.where(slot >= 0, slot, ~slot)
    token = torch.arange(c["T"], device=row.device).repeat_interleave(c["k"])
    expert = torch.searchsorted(off[1:].contiguous(), row.int(), right=True)
    at = expert * s["most"] + row - off[:-1].long()[expert]
    a = torch.zeros((E * s["most"], K), dtype=torch.float32, device=row.device)
    a[at] = torch.where((slot >= 0)[:, None], xq[token], torch.zeros_like(xq[:1]))
    raw = s["sb"].view(E, -1)
    C4 = (K // 32 + 3) // 4
    sb = raw.view(E, -1, C4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1, 4 * C4)[:, :N, :K // 32]
    full = torch.bmm(a.view(E, s["most"], K), _dequantized4(s["qb"], sb).transpose(1, 2)).view(-1, N)
    out = torch.empty((row.numel(), N), dtype=DTYPES[c["out"]], device=row.device)
    out[row] = full[at].to(out.dtype)
    return {"rows": out, "slot_row": slot_row}


def run(s):
    if not own:
        return _plain(s)
    from mxfp8_block_scaled_07_b200 import mx

    c = s["c"]
    op = c["op"]
    if op == "route":
        ids, w = mx.route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                          topk_groups=c["topk_groups"], group_score=c["group_score"], renormalize=c["renorm"],
                          scale=c["scale"])
        if not c["train"]:
            return {"ids": ids, "weights": w}
        d = mx.route_backward(s["d_weights"], s["logits"], ids, score=c["score"], renormalize=c["renorm"],
                              scale=c["scale"])
        return {"ids": ids, "weights": w, "d_logits": d}
    if op == "dispatch":
        off, slot_row, counts = mx.route_plan(s["ids"], c["E"])
        q, sc = mx.dispatch_quantize(s["x"], slot_row, off)
        return {"offsets": off, "slot_row": slot_row, "counts": counts, "codes": q.view(torch.float8_e4m3fn),
                "scales": sc.view(torch.float8_e8m0fnu)}
    if op == "combine":
        y = mx.combine(s["rows"], s["slot_row"], s["weights"])
        if not c["train"]:
            return {"y": y}
        d_rows, dw = mx.combine_backward(s["dy"], s["rows"], s["slot_row"], s["weights"])
        return {"y": y, "d_rows": d_rows, "d_weights": dw}
    if op == "quantize":
        q, sc, qc, scc = mx.quantize_fp4(s["x"], colwise=c["col"])
        out = {"scales_row": sc.view(torch.float8_e8m0fnu), "values_row": mx.dequantize_fp4(q, sc)}
        if c["col"]:
            out["scales_col"], out["values_col"] = scc.view(torch.float8_e8m0fnu), mx.dequantize_fp4(qc, scc)
        return out
    if op == "product":
        return mx.gemm_fp4(s["qa"], s["sa"], s["qb"], s["sb"], out_dtype=DTYPES[c["out"]])
    off, slot_row, _ = mx.route_plan(s["ids"], c["E"])
    q, sc = mx.dispatch_quantize(s["x"], slot_row, off, fmt="mxfp4")
    rows = mx.grouped_gemm_fp4(q, sc, s["qb"], s["sb"], off, out_dtype=DTYPES[c["out"]])
    return {"rows": rows, "slot_row": slot_row}


# ---- definitions in fp64 -----------------------------------------------------------------------------------------------

# The magnitudes a code of each format stands for, in code order.
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(x, grid):
    """Every fp64 value's nearest member of the grid (magnitudes in code order), ties to the even code, beyond the end
    to the largest."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    at = torch.searchsorted(mid, a)
    tie = (at < mid.numel()) & (a == mid[at.clamp(max=mid.numel() - 1)]) & (at % 2 == 1)
    return torch.copysign(grid[at + tie.long()], x)


def _microscaled(x, grid, emax):
    """(values on the grid, block scales 2^e, their product) of fp64 input, blocks of 32 along the last axis. An
    all-zero block takes the smallest scale, 2^-127."""
    b = x.reshape(-1, 32)
    power = torch.tensor([2.0 ** i for i in range(-150, 129)], dtype=torch.float64, device=x.device)
    e = torch.searchsorted(power, b.abs().amax(dim=1), right=True) - 151 - emax      # floor(log2 amax) - emax
    scale = power[e.clamp(min=-127) + 150][:, None]
    v = _nearest(b / scale, grid)
    return v.reshape(x.shape), scale.reshape(*x.shape[:-1], -1), (v * scale).reshape(x.shape)


def _layout64(scale, index, rows, pad=2.0 ** -127):
    """Scales [n, kblocks] put at rows `index` of the tensor-core layout of `rows` (a multiple of 128) rows; pads 2^-127."""
    C = scale.shape[1]
    ct = (C + 3) // 4
    out = torch.full((rows * 4 * ct,), pad, dtype=torch.float64, device=scale.device)
    r, col = index[:, None], torch.arange(C, device=scale.device)[None, :]
    out[((r // 128) * ct + col // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + col % 4] = scale
    return out


def _decoded64(q, scales, rows, N=None):
    """fp64 values of packed codes [n, K/2] whose scales lie at rows `rows` of a layout."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=q.device)
    v = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = table[(q & 15).long()], table[(q >> 4).long()]
    C = v.shape[1] // 32
    ct = (C + 3) // 4
    r, col = rows[:, None], torch.arange(C, device=q.device)[None, :]
    byte = scales[((r // 128) * ct + col // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + col % 4]
    return (v.view(-1, C, 32) * byte.view(torch.float8_e8m0fnu).double()[:, :, None]).view(v.shape)


def exact(c, seed):
    s, op = prepare(c, seed), c["op"]
    if op == "route":
        ids = _route(s["logits"], s["bias"], c)[0].long()      # whole numbers: only the weights have a value in fp64
        x = s["logits"].double().requires_grad_(True)
        got = ids >= 0
        z = torch.gather(x, 1, ids.clamp(min=0))
        z = torch.where(got, z, torch.full_like(z, float("-inf")))
        some = got.any(dim=1)
        if c["score"] == "sigmoid":
            logs = torch.nn.functional.logsigmoid(z[some])
        else:
            logs = z[some] - torch.logsumexp(x[some], dim=1, keepdim=True)
        if c["renorm"]:
            logs = logs - torch.logsumexp(logs, dim=1, keepdim=True)
        w = torch.zeros(ids.shape, dtype=torch.float64, device=x.device)
        w[some] = c["scale"] * torch.where(got[some], torch.exp(logs), torch.zeros_like(logs))
        out = {"ids": None, "weights": w.detach()}
        if c["train"]:
            (d,) = torch.autograd.grad(torch.where(got, w * s["d_weights"].double(), torch.zeros_like(w)).sum(), x)
            out["d_logits"] = torch.nan_to_num(d, nan=0.0)      # a masked entry: 0 times an infinity
        return out
    if op == "dispatch":
        T, E, k, K = c["T"], c["E"], c["k"], c["K"]
        ids = s["ids"].reshape(-1).long()
        order = torch.sort(torch.where(ids < 0, E, ids), stable=True).indices
        v, scale, _ = _microscaled(s["x"].double(), E4M3, 8)
        live = (ids[order] >= 0).double()[:, None]
        group = torch.where(ids[order] < 0, E - 1, ids[order])
        sizes = torch.bincount(group, minlength=E)
        starts = torch.cumsum(sizes, 0) - sizes
        tiles = (sizes + 127) // 128
        at = ((torch.cumsum(tiles, 0) - tiles) * 128)[group] + torch.arange(T * k, device=ids.device) - starts[group]
        rows = (T * k + 127 * min(E, T * k)) // 128 * 128
        sc = torch.where(live > 0, scale[order // k], torch.full_like(scale[:1], 2.0 ** -127))
        return {"offsets": None, "slot_row": None, "counts": None, "codes": v[order // k] * live,
                "scales": _layout64(sc, at, rows)}
    if op == "combine":
        T, k, N = c["T"], c["k"], c["N"]
        token = torch.arange(T, device="cuda").repeat_interleave(k)
        slot, w = s["slot_row"].reshape(-1).long(), s["weights"].reshape(-1).double()
        live = torch.nonzero(slot >= 0).reshape(-1)
        y = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        y.index_add_(0, token[live], s["rows"][slot[live]].double() * w[live, None])
        if not c["train"]:
            return {"y": y}
        d_rows = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
        d_rows[slot[live]] = s["dy"].double()[token[live]] * w[live, None]
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dw[live] = torch.einsum("rn,rn->r", s["rows"][slot[live]].double(), s["dy"][token[live]].double())
        return {"y": y, "d_rows": d_rows, "d_weights": dw.view(T, k)}
    if op == "quantize":
        out = {}
        for way in ("row", "col") if c["col"] else ("row",):
            x = s["x"].double() if way == "row" else s["x"].double().t().contiguous()
            _, scale, value = _microscaled(x, E2M1, 2)
            n = x.shape[0]
            out["scales_" + way] = _layout64(scale, torch.arange(n, device=x.device), (n + 127) // 128 * 128)
            out["values_" + way] = value
        return out
    if op == "product":
        a = _decoded64(s["qa"], s["sa"], torch.arange(c["M"], device="cuda"))
        b = _decoded64(s["qb"], s["sb"], torch.arange(c["N"], device="cuda"))
        return torch.einsum("mk,nk->mn", a, b)
    T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
    ids = s["ids"].reshape(-1).long()
    order = torch.sort(torch.where(ids < 0, E, ids), stable=True).indices
    x = _microscaled(s["x"].double(), E2M1, 2)[2]
    out = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
    pad = (N + 127) // 128 * 128
    for g in range(E):
        mine = torch.nonzero(ids[order] == g).reshape(-1)
        b = _decoded64(s["qb"][g], s["sb"], g * pad + torch.arange(N, device="cuda"))
        out[mine] = x[order[mine] // k] @ b.t()
    return {"rows": out, "slot_row": None}
