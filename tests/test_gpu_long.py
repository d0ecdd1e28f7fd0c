"""MXFP4 and routing calls whose offsets pass 2^31 elements: the last rows are what a call on those rows alone gives, bit for
bit (every row is computed by itself, in the same order). Up to 10 GB on the device at a time."""
import gc

import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu

LAST = 256


@pytest.fixture(autouse=True)
def release():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def tail(rows, cols, seed, dtype=torch.bfloat16):
    """[rows, cols], zeros but for the last LAST rows."""
    x = torch.zeros((rows, cols), dtype=dtype, device="cuda")
    x[-LAST:] = torch.randn((LAST, cols), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    return x


@pytest.mark.parametrize("renormalize", [True, False])
def test_route(renormalize):
    T, E, k = 2_200_000, 1024, 4
    x = tail(T, E, 1)
    ids, w = mx.route(x, k, renormalize=renormalize)
    few = x[-LAST:].contiguous()
    ids1, w1 = mx.route(few, k, renormalize=renormalize)
    assert torch.equal(ids[-LAST:], ids1) and torch.equal(w[-LAST:], w1)
    d = torch.ones_like(w)
    d[-LAST:] = torch.arange(LAST * k, device="cuda").view(LAST, k) / 7.0
    g = mx.route_backward(d, x, ids, renormalize=renormalize)
    assert torch.equal(g[-LAST:], mx.route_backward(d[-LAST:].contiguous(), few, ids1, renormalize=renormalize))


def test_dispatch():
    T, k, E, K = 136_000, 8, 64, 2048
    x = tail(T, K, 2)
    ids = torch.stack([torch.randperm(E, device="cuda")[:k] for _ in range(32)]).repeat(T // 32, 1).to(torch.int32)
    ids[-LAST:] = E - 1 - torch.arange(k, device="cuda", dtype=torch.int32)
    off, slot_row, _ = mx.route_plan(ids, E)
    for fmt, one in (("mxfp8", lambda v: mx.quantize(v)), ("mxfp4", lambda v: mx.quantize_fp4(v))):
        q, s = mx.dispatch_quantize(x, slot_row, off, fmt)
        want = one(x[-LAST:].contiguous())[0]
        for j in range(k):
            assert torch.equal(q[slot_row[-LAST:, j].long()], want)
        del q, s


def test_combine_and_gradients():
    R, N, T, k = 1_100_800, 2048, 200, 3
    c = tail(R, N, 3)
    g = torch.Generator().manual_seed(4)
    # One row per token, the other slots' padding row (~slot_row) outside: no row is named twice.
    near = torch.full((T, k), -2 ** 31, dtype=torch.int32, device="cuda")
    near[:, 0] = torch.randperm(LAST, generator=g)[:T].to(torch.int32).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    far = torch.where(near >= 0, near + (R - LAST), near)
    few = c[-LAST:].contiguous()
    y = mx.combine(c, far, w)
    assert torch.equal(y, mx.combine(few, near, w)) and y.any()
    dy = torch.randn((T, N), generator=g).cuda()
    d_c, d_w = mx.combine_backward(dy, c, far, w)
    d_c1, d_w1 = mx.combine_backward(dy, few, near, w)
    assert torch.equal(d_w, d_w1) and torch.equal(d_c[-LAST:], d_c1)
    del d_c, d_c1
    # Many tokens: the output's offsets.
    one = torch.arange(R, dtype=torch.int32, device="cuda").view(R, 1)
    y = mx.combine(c, one)
    assert torch.equal(y[-LAST:], few)


def test_quantize_and_dequantize():
    M, K = 1_100_800, 2048
    x = tail(M, K, 5)
    few = x[-LAST:].contiguous()
    q, s, qc, sc = mx.quantize_fp4(x, True, True, swizzle=False)
    q1, s1, qc1, sc1 = mx.quantize_fp4(few, True, True, swizzle=False)
    assert torch.equal(q[-LAST:], q1) and torch.equal(s[-LAST:], s1)
    assert torch.equal(qc[:, -LAST // 2:], qc1) and torch.equal(sc[:, -LAST // 32:], sc1)
    back = mx.dequantize_fp4(q, s, swizzled=False)
    assert torch.equal(back[-LAST:], mx.dequantize_fp4(q1, s1, swizzled=False))


def codes(rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    return mx.quantize_fp4(torch.randn((rows, K), generator=g).to(torch.bfloat16).cuda())[:2]


def test_product_outputs():
    N, K = 32_768, 64
    qb, sb = codes(N, K, 6)
    M = 70_016
    qa, sa = codes(M, K, 7)
    c = mx.gemm_fp4(qa, sa, qb, sb)
    kt = sa.numel() // M                            # scale bytes per row: whole 128-row tiles follow one another
    assert torch.equal(c[-128:], mx.gemm_fp4(qa[-128:].contiguous(), sa[-128 * kt:].contiguous(), qb, sb))
    del c
    # Row strides of 2^26 elements and more: few rows, and few rows per group.
    n = 384
    qb, sb = qb[:n].contiguous(), sb[:n * kt].contiguous()
    out = torch.empty(9 * 2 ** 28 + n, dtype=torch.bfloat16, device="cuda").as_strided((10, n), (2 ** 28, 1))
    want = mx.gemm_fp4(qa[:10].contiguous(), sa[:128 * kt].contiguous(), qb, sb)
    assert torch.equal(mx.gemm_fp4(qa[:10].contiguous(), sa[:128 * kt].contiguous(), qb, sb, out=out), want)
    del out
    off = torch.tensor([0, 17, 40], dtype=torch.int32, device="cuda")
    out = torch.empty(39 * 2 ** 26 + n // 2, dtype=torch.bfloat16, device="cuda").as_strided((40, n // 2), (2 ** 26, 1))
    a = (qa[:40].contiguous(), sa[:256 * kt].contiguous(), qb.view(2, n // 2, K // 2), torch.cat([sb[:256 * kt], sb[:256 * kt]]), off)
    assert torch.equal(mx.grouped_gemm_fp4(*a, out=out), mx.grouped_gemm_fp4(*a))
