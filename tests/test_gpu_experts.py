"""GPU parity of dispatch, combine and combine's gradient, and the whole expert layer run together.

Tolerances (u = 2^-24; h = half a step of the output type, 2^-24 fp32, 2^-8 BF16): combine adds k terms with fused
multiply-adds, k u of sum |w c|, then one rounding; d_rows is one fp32 product and one rounding, u + h of the value;
d_weights' dot product over N columns runs in per-lane chains of ceil(N / 2048) * 8 terms, joined over 32 lanes and 8
warps, fewer than N / 256 + 32 roundings of sum |dy c|."""
import numpy as np
import pytest
import torch

import oracle
import plain
from helpers import assert_gemm_close, to_np
from mxfp8_block_scaled_07_b200 import mx, synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def choose(T, k, E, seed, dropped):
    g = np.random.default_rng(seed)
    ids = np.argsort(g.random((T, E)) - 0.7 * np.arange(E) / E, axis=1)[:, :k]
    if dropped:
        ids[g.random((T, k)) < 0.2] = -1
        ids[T // 2] = -1
    return ids


def cuda32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 32), (1, 8, 128, 64), (13, 8, 128, 2048), (40, 3, 5, 96), (300, 2, 4, 160), (129, 4, 16, 1056),
                                     (70, 1, 3, 4096), (33, 40, 60, 64)])
def test_dispatch(T, k, E, K, dropped, fmt):
    ids = choose(T, k, E, T + E, dropped)
    off, slot_row, _ = plain.plan(ids, E)
    x = synth.normal_bf16((T, K), seed=K, outlier_frac=0.01, outlier_scale=100.0)
    q, s = mx.dispatch_quantize(x.cuda(), cuda32(slot_row), cuda32(off), fmt)
    if fmt == "mxfp8":
        codes, sc = oracle.quantize_rowwise(x)
    else:
        c4, sc = plain.quantize_fp4(x.double().numpy())
        codes = plain.pack(c4)
    want, raw = np.zeros((T * k, codes.shape[1]), np.uint8), np.zeros((T * k, K // 32), np.uint8)
    for t, j in np.ndindex(T, k):
        if slot_row[t, j] >= 0:
            want[slot_row[t, j]], raw[slot_row[t, j]] = codes[t], sc[t]
    assert np.array_equal(to_np(q), want)
    assert np.array_equal(to_np(s), plain.grouped_layout(raw, off, mx.grouped_scale_bytes_bound(T * k, E, K // 32)))


def test_dispatch_strided_and_special_input():
    T, k, E, K = 60, 2, 7, 96
    x = synth.special_bf16((T, K), seed=1)
    ids = choose(T, k, E, 3, True)
    off, slot_row, _ = plain.plan(ids, E)
    for pad, start in ((8, 0), (0, 8), (16, 0)):
        flat = torch.zeros(T * (K + pad) + start, dtype=torch.bfloat16, device="cuda")
        d = flat[start:].view(T, K + pad)[:, :K]
        d.copy_(x)
        q, s = mx.dispatch_quantize(d, cuda32(slot_row), cuda32(off))
        codes, sc = oracle.quantize_rowwise(x)
        got = to_np(q)
        for t, j in np.ndindex(T, k):
            if slot_row[t, j] >= 0:
                assert np.array_equal(got[slot_row[t, j]], codes[t])
            else:
                assert not got[~slot_row[t, j]].any()


def test_dispatch_skips_rows_and_places_outside_its_buffers():
    """Rows past T * topk, offsets that are no partition: nothing outside the outputs is touched."""
    T, k, E, K = 8, 2, 3, 64
    x = synth.normal_bf16((T, K), seed=2).cuda()
    n, ns = T * k * K, mx.grouped_scale_bytes_bound(T * k, E, K // 32)
    for rows, off in ((np.full((T, k), 16), [0, 5, 5, 16]), (np.full((T, k), 2 ** 31 - 1), [0, 5, 5, 16]),
                      (np.full((T, k), -2 ** 31), [0, 5, 5, 16]), (np.arange(16).reshape(T, k), [0, 2 ** 31 - 1, 5, 16]),
                      (np.arange(16).reshape(T, k), [-2 ** 31, -5, 3, -1]), (np.arange(16).reshape(T, k), [9, 9, 9, 9])):
        buf, sbuf = (torch.full((m + 64,), 0xA5, dtype=torch.uint8, device="cuda") for m in (n, ns))
        mx.dispatch_quantize(x, cuda32(rows), cuda32(np.array(off)), out=(buf[32:32 + n].view(T * k, K), sbuf[32:32 + ns]))
        for b, m in ((buf, n), (sbuf, ns)):
            assert torch.all(b[:32] == 0xA5) and torch.all(b[32 + m:] == 0xA5)


@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ct", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,E,N", [(1, 1, 1, 1), (3, 8, 16, 256), (13, 8, 128, 2048), (50, 3, 5, 100), (21, 5, 8, 2300), (40, 40, 60, 33)])
def test_combine_and_gradients(T, k, E, N, ct, yt):
    ids = choose(T, k, E, T + N, True)
    _, slot_row, _ = plain.plan(ids, E)
    g = torch.Generator().manual_seed(N)
    rows, dy = torch.randn((T * k, N), generator=g).to(ct), torch.randn((T, N), generator=g).to(yt)
    w = torch.randn((T, k), generator=g)
    sr = cuda32(slot_row)
    r64, d64, w64 = (t.double().numpy() for t in (rows, dy, w))
    for weights, v in ((w.cuda(), w64), (None, np.ones((T, k)))):
        y = mx.combine(rows.cuda(), sr, weights, out_dtype=yt)
        ref, size = plain.combine(r64, slot_row, v)
        assert y.dtype == yt
        assert np.all(np.abs(to_np(y.double()) - ref) <= (k + 1) * U * size * (1 + 2.0 ** -8) + HALF[yt] * np.abs(ref))
    d_rows, dw = mx.combine_backward(dy.cuda(), rows.cuda(), sr, w.cuda())
    ref_rows, ref_w, size = plain.combine_backward(d64, r64, slot_row, w64)
    assert d_rows.dtype == ct
    assert np.all(np.abs(to_np(d_rows.double()) - ref_rows) <= (U + HALF[ct]) * np.abs(ref_rows) * (1 + 2.0 ** -8))
    assert np.all(np.abs(to_np(dw) - ref_w) <= (N / 256 + 48) * U * size)
    only_rows, none = mx.combine_backward(dy.cuda(), rows.cuda(), sr, w.cuda(), need_weights=False)
    assert none is None and torch.equal(only_rows, d_rows)
    # The gradient of a plain gather (weights 1) and its transpose, the plain sum, are each other's.
    ones, _ = mx.combine_backward(dy.cuda(), rows.cuda(), sr, None, need_weights=False)
    live = slot_row[slot_row >= 0]
    tok = np.repeat(np.arange(T), k).reshape(T, k)[slot_row >= 0]
    assert torch.equal(ones[cuda32(live).long()], dy.cuda().to(ct)[cuda32(tok).long()])


def test_combine_strides_and_rows_outside():
    T, k, N = 9, 2, 40
    g = torch.Generator().manual_seed(1)
    wide = torch.randn((18, N + 3), generator=g).cuda()
    rows = wide[:, 1:1 + N]                                       # unaligned rows: element accesses
    sr = np.arange(18).reshape(T, k)
    sr[0], sr[1, 0], sr[2, 1] = -1, 18, 2 ** 31 - 1               # no expert; past the rows
    out = torch.full((T, N + 7), 5.0, device="cuda")
    mx.combine(rows, cuda32(sr), None, out=out[:, :N])
    ref, _ = plain.combine(rows.cpu().double().numpy(), sr, np.ones((T, k)))
    assert np.allclose(to_np(out[:, :N]), ref, rtol=1e-6, atol=1e-6) and torch.all(out[:, N:] == 5.0)
    assert not out[0, :N].any()
    dy = torch.randn((T, N), generator=g).cuda()
    before = torch.full((18, N), 5.0, device="cuda")
    _, dw = mx.combine_backward(dy, rows, cuda32(sr), None, out=(before, torch.empty((T, k), device="cuda")))
    assert torch.all(before[2] == 5.0) and torch.all(before[5] == 5.0)      # rows that no slot names
    assert not dw[0].any() and dw[1, 0] == 0 and dw[2, 1] == 0


# ---- together -----------------------------------------------------------------------------------------

def interleave(w):
    G, n2, K = w.shape
    return w.view(G, 2, n2 // 256, 128, K).permute(0, 2, 1, 3, 4).reshape(G, n2, K).contiguous()


def moe_inputs(T, E, H, n, seed=0):
    return (synth.normal_bf16((T, H), seed=seed), synth.normal_bf16((T, E), seed=seed + 1),
            synth.normal_bf16((E, 2 * n, H), std=0.05, seed=seed + 2), synth.normal_bf16((E, H, n), std=0.05, seed=seed + 3))


def moe_mxfp8(x, logits, q1, q2, E, k, n):
    """One MoE layer's forward pass through the library alone."""
    H = x.shape[1]
    ids, w = mx.route(logits, k)
    off, slot_row, _ = mx.route_plan(ids, E)
    qa, sa = mx.dispatch_quantize(x, slot_row, off)
    rows = x.shape[0] * k
    h = (torch.empty((rows, n), dtype=torch.uint8, device=x.device),
         torch.zeros(mx.grouped_scale_bytes_bound(rows, E, n // 32), dtype=torch.uint8, device=x.device))
    mx.grouped_gemm_swiglu_quant(qa, sa, q1[0], q1[1], off, None, out=h)
    c = mx.grouped_gemm(h[0], h[1], q2[0], q2[1], off)
    return ids, w, off, slot_row, h, c, mx.combine(c, slot_row, w)


def quantized_weights(w):
    G, N, K = w.shape
    q, s, _, _ = mx.quantize(w.reshape(G * N, K))
    return q.view(G, N, K), s


@pytest.mark.parametrize("T,masked", [(1, False), (200, False), (64, True)])
def test_moe_layer_mxfp8(T, masked):
    """Router to output through the library; the layer's output against fp64 from the operands the products read
    (their codes), with padding tokens whose logits are all -inf."""
    E, k, H, n = 16, 4, 256, 128
    x, logits, w1, w2 = moe_inputs(T, E, H, n)
    if masked:
        logits[T - 5:] = float("-inf")
    q1, q2 = quantized_weights(interleave(w1).cuda()), quantized_weights(w2.cuda())
    ids, w, off, slot_row, h, c, y = moe_mxfp8(x.cuda(), logits.cuda(), q1, q2, E, k, n)
    assert mx.device_error() == 0
    want, w64 = plain.route(logits.double().numpy(), k)
    assert np.array_equal(to_np(ids), want)
    o, s, counts = plain.plan(want, E)
    assert np.array_equal(to_np(off), o) and np.array_equal(to_np(slot_row), s)
    # The down product against fp64 of the activation's own codes, expert by expert.
    hq, hs = to_np(h[0]), to_np(h[1])
    q2n, s2n = oracle.quantize_rowwise(w2.reshape(E * H, n))
    tile = 0
    ref, size = np.zeros((T * k, H)), np.zeros((T * k, H))
    for g in range(E):
        m = o[g + 1] - o[g]
        r, cidx = np.arange(m)[:, None], np.arange(n // 32)[None, :]
        at = ((tile + r // 128) * (n // 128) + cidx // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + cidx % 4
        tile += (m + 127) // 128
        if m:
            ref[o[g]:o[g + 1]], size[o[g]:o[g + 1]] = oracle.gemm(hq[o[g]:o[g + 1]], np.ascontiguousarray(hs[at]),
                                                                  q2n[g * H:(g + 1) * H], s2n[g * H:(g + 1) * H])
    assert_gemm_close(to_np(c.float()), ref, size, True, "down product")
    out, total = plain.combine(to_np(c.double()), s, to_np(w.double()))
    assert np.all(np.abs(to_np(y.double()) - out) <= (k + 1) * U * total + 2.0 ** -8 * np.abs(out))
    if masked:
        assert not y[T - 5:].any() and not c[cuda32(~s[T - 5:]).long()].any()


def test_moe_product_mxfp4():
    """Router, plan, MXFP4 dispatch and grouped product against fp64 on the values of the codes."""
    T, E, k, H, N = 150, 8, 3, 288, 200
    x, logits, _, _ = moe_inputs(T, E, H, 128, seed=5)
    wt = synth.normal_bf16((E, N, H), std=0.05, seed=9)
    qb = [mx.quantize_fp4(wt[e].cuda()) for e in range(E)]
    ids, w = mx.route(logits.cuda(), k, "sigmoid", groups=4, topk_groups=2, group_score="top2")
    off, slot_row, _ = mx.route_plan(ids, E)
    qa, sa = mx.dispatch_quantize(x.cuda(), slot_row, off, "mxfp4")
    c = mx.grouped_gemm_fp4(qa, sa, torch.stack([q[0] for q in qb]), torch.cat([q[1] for q in qb]), off, torch.float32)
    y = mx.combine(c, slot_row, w)
    assert mx.device_error() == 0

    def val(t):
        code, s = plain.quantize_fp4(t.double().numpy())
        return plain.values_fp4(plain.pack(code), s)

    xv, ids_n = val(x), to_np(ids)
    ref, size = np.zeros((T, N)), np.zeros((T, N))
    for t, j in np.ndindex(T, k):
        wv = val(wt[ids_n[t, j]])
        ref[t] += float(w[t, j]) * (wv @ xv[t])
        size[t] += float(w[t, j]) * (np.abs(wv) @ np.abs(xv[t]))
    assert np.all(np.abs(to_np(y) - ref) <= (1e-5 + 8 * U) * size)


def test_layer_replays_in_a_cuda_graph_and_on_another_stream():
    """The calls allocate nothing and wait for nothing: captured once and replayed on new inputs (other tokens, other
    choices, other loads per expert) they give what eager calls give; so does a run on a side stream."""
    T, E, k, H, n = 96, 16, 4, 256, 128
    x, logits, w1, w2 = (t.cuda() for t in moe_inputs(T, E, H, n))
    q1, q2 = quantized_weights(interleave(w1)), quantized_weights(w2)
    dy = synth.normal_bf16((T, H), seed=8).cuda()

    def step():
        ids, w, off, slot_row, h, c, y = moe_mxfp8(x, logits, q1, q2, E, k, n)
        d_c, d_w = mx.combine_backward(dy, c, slot_row, w)
        return ids, w, off, slot_row, c, y, d_c, d_w, mx.route_backward(d_w, logits, ids)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (21, 22):
        a, b, _, _ = moe_inputs(T, E, H, n, seed=seed)
        x.copy_(a)
        logits.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for u, v in zip(got, step()):
            assert torch.equal(u, v)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step()
        side.synchronize()
        for u, v in zip(got, other):
            assert torch.equal(u, v)


class Layer:
    """An MXFP4 expert layer whose every step writes into buffers of its own that each pass uses again."""

    def __init__(self, T, k, E, H, N, seed):
        g = torch.Generator().manual_seed(seed)
        self.k, self.E = k, E
        self.inputs = [(torch.randn((T, H), generator=g).to(torch.bfloat16).cuda(),
                        torch.randn((T, E), generator=g).cuda(), torch.randn((E * N, H), generator=g).to(torch.bfloat16).cuda())
                       for _ in range(3)]
        self.x, self.logits, self.w = (torch.empty_like(v) for v in self.inputs[0])
        self.qw = mx.quantize_fp4(self.w)
        self.wq = self.qw[0].view(E, N, H // 2)
        self.choice = mx.route(self.logits.zero_(), k)
        self.part = mx.route_plan(self.choice[0], E)
        self.q = mx.dispatch_quantize(self.x.zero_(), self.part[1], self.part[0], "mxfp4")
        self.rows = torch.empty((T * k, N), device="cuda")
        self.y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        self.grads = (torch.empty_like(self.rows), torch.empty_like(self.choice[1]))
        self.d_logits = torch.empty_like(self.logits)
        self.dense = torch.empty((min(T, 48), E * N), device="cuda")
        self.back = torch.empty_like(self.x[:len(self.dense)])

    def steps(self, i):
        """The calls of pass i, in order."""
        for a, b in zip((self.x, self.logits, self.w), self.inputs[i % len(self.inputs)]):
            yield lambda a=a, b=b: a.copy_(b)
        yield lambda: mx.quantize_fp4(self.w, out=self.qw)
        yield lambda: mx.route(self.logits, self.k, out=self.choice)
        yield lambda: mx.route_plan(self.choice[0], self.E, out=self.part)
        yield lambda: mx.dispatch_quantize(self.x, self.part[1], self.part[0], "mxfp4", out=self.q)
        yield lambda: mx.grouped_gemm_fp4(self.q[0], self.q[1], self.wq, self.qw[1], self.part[0], out=self.rows)
        yield lambda: mx.combine(self.rows, self.part[1], self.choice[1], out=self.y)
        yield lambda: mx.combine_backward(self.y, self.rows, self.part[1], self.choice[1], out=self.grads)
        yield lambda: mx.route_backward(self.grads[1], self.logits, self.choice[0], out=self.d_logits)
        qx = mx.quantize_fp4(self.x[:len(self.dense)])
        yield lambda: mx.gemm_fp4(qx[0], qx[1], self.qw[0], self.qw[1], out=self.dense)
        yield lambda: mx.dequantize_fp4(qx[0], qx[1], out=self.back)

    def answers(self):
        return [t.clone() for t in (*self.choice, *self.part, *self.q, self.rows, self.y, *self.grads, self.d_logits, self.dense, self.back)]


# T * k: a plan of one block, of a cluster, with a counting kernel; grouped products of few and of many rows per expert.
@pytest.mark.parametrize("T,k,E,H,N", [(24, 2, 64, 256, 128), (700, 8, 16, 512, 256), (9000, 4, 16, 128, 256)])
def test_calls_back_to_back_wait_for_one_another(T, k, E, H, N):
    """Kernels become resident before the ones in front of them have ended: passes without a pause, over the same buffers and
    with changing inputs, give what passes give that wait after every call; so does a captured pass, also where a
    second stream joins in its middle."""
    layer = Layer(T, k, E, H, N, T)
    want = []
    for i in range(3):
        for step in layer.steps(i):
            step()
            torch.cuda.synchronize()
        want.append(layer.answers())
    got = []
    for i in range(24):
        for step in layer.steps(i):
            step()
        got.append(layer.answers())
    for i, answers in enumerate(got):
        for a, b in zip(answers, want[i % 3]):
            assert torch.equal(a, b)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    source = [torch.empty_like(v) for v in layer.inputs[0]]
    layer.inputs.append(tuple(source))
    with torch.cuda.graph(graph):
        for n, step in enumerate(layer.steps(3)):
            if n % 3 == 2:                       # every third call on another stream
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    step()
                torch.cuda.current_stream().wait_stream(side)
            else:
                step()
    layer.inputs.pop()
    for i in range(6):
        for a, b in zip(source, layer.inputs[i % 3]):
            a.copy_(b)
        graph.replay()
        for a, b in zip(layer.answers(), want[i % 3]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("ct,yt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,k,E,N", [(700, 1, 3, 96), (333, 9, 40, 200), (501, 2, 7, 500), (258, 8, 16, 1000), (129, 3, 5, 1024)])
def test_combine_and_gradients_of_narrow_rows(T, k, E, N, ct, yt):
    """Several tokens per block: rows of one, two, four and more pieces, tokens that do not fill the last block."""
    test_combine_and_gradients(T, k, E, N, ct, yt)
