"""GPU parity of the MXFP4 operators: quantization and dequantization bit for bit, dense and grouped products within
the library's GEMM bound (|c - ref| <= 1e-5 sum |a_k b_k|, + 2^-8 |ref| for BF16 output) of fp64."""
import numpy as np
import pytest
import torch

import oracle
import plain
from helpers import assert_gemm_close, scale_positions, to_np
from mxfp8_block_scaled_07_b200 import mx, synth

pytestmark = pytest.mark.gpu


def f64(x):
    return x.to(torch.float64).numpy()


def assert_quantized(x, q, s, swizzle, what):
    """x: float64 [M, K] as the direction sees it."""
    code, sb = plain.quantize_fp4(x)
    assert np.array_equal(to_np(q), plain.pack(code)), f"{what}: codes"
    want = oracle.swizzle(sb) if swizzle else sb
    assert np.array_equal(to_np(s).reshape(-1), want.reshape(-1)), f"{what}: scales"


SHAPES = [(1, 32), (3, 64), (127, 96), (128, 128), (130, 160), (256, 512), (300, 416), (1, 4096), (1000, 1056)]


@pytest.mark.parametrize("swizzle", [True, False])
@pytest.mark.parametrize("M,K", SHAPES)
def test_rowwise(M, K, swizzle):
    x = synth.normal_bf16((M, K), seed=M + K, outlier_frac=0.01, outlier_scale=100.0)
    q, s, _, _ = mx.quantize_fp4(x.cuda(), swizzle=swizzle)
    assert_quantized(f64(x), q, s, swizzle, "rowwise")


@pytest.mark.parametrize("row", [True, False])
@pytest.mark.parametrize("swizzle", [True, False])
@pytest.mark.parametrize("M,K", [(32, 32), (96, 64), (128, 128), (160, 288), (544, 96), (32, 1312)])
def test_columnwise(M, K, swizzle, row):
    x = synth.normal_bf16((M, K), seed=M + K, outlier_frac=0.01, outlier_scale=100.0)
    q, s, qc, sc = mx.quantize_fp4(x.cuda(), rowwise=row, colwise=True, swizzle=swizzle)
    if row:
        assert_quantized(f64(x), q, s, swizzle, "rowwise")
    assert_quantized(f64(x).T.copy(), qc, sc, swizzle, "columnwise")


@pytest.mark.parametrize("seed", range(3))
def test_adversarial_patterns(seed):
    """Every exponent, signed zeros, subnormals, blocks of zeros, NaN and infinities."""
    x = synth.special_bf16((320, 512), seed=seed)
    q, s, qc, sc = mx.quantize_fp4(x.cuda(), colwise=True)
    assert_quantized(f64(x), q, s, True, "rowwise")
    assert_quantized(f64(x).T.copy(), qc, sc, True, "columnwise")


def test_every_bf16_pattern():
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for x in (bits.view(2048, 32), bits.view(32, 2048).t().contiguous()):
        q, s, _, _ = mx.quantize_fp4(x.cuda(), swizzle=False)
        assert_quantized(f64(x), q, s, False, "patterns")


@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 0), (0, 8), (24, 8)])
def test_strided_and_offset_input(pad, offset):
    """Row strides that are no multiple of 32 bytes, and a start that is 16- but not 32-byte aligned."""
    M, K = 200, 192
    flat = synth.normal_bf16((M * (K + pad) + offset,), seed=5)
    x = flat[offset:].view(M, K + pad)[:, :K]
    d = flat.cuda()[offset:].view(M, K + pad)[:, :K]
    q, s, _, _ = mx.quantize_fp4(d)
    assert_quantized(f64(x), q, s, True, "strided")


def test_nothing_outside_the_outputs_is_written():
    M, K = 130, 96
    x = synth.normal_bf16((M, K), seed=1).cuda()
    n, ns = M * K // 2, mx.swizzled_scale_bytes(M, K // 32)
    buf, sbuf = (torch.full((m + 64,), 0xA5, dtype=torch.uint8, device="cuda") for m in (n, ns))
    mx.quantize_fp4(x, out=(buf[32:32 + n].view(M, K // 2), sbuf[32:32 + ns], None, None))
    for b, m in ((buf, n), (sbuf, ns)):
        assert torch.all(b[:32] == 0xA5) and torch.all(b[32 + m:] == 0xA5)


@pytest.mark.parametrize("swizzled", [True, False])
@pytest.mark.parametrize("M,K,pad", [(1, 32, 0), (130, 96, 8), (257, 160, 0)])
def test_dequantize(M, K, pad, swizzled):
    """Every code under scales 0 to 252 and 255 (above 252 a product may pass BF16's range)."""
    g = np.random.default_rng(M)
    q = g.integers(0, 256, (M, K // 2), dtype=np.uint8)
    raw = g.integers(0, 254, (M, K // 32), dtype=np.uint8)
    raw[raw == 253] = 255
    s = oracle.swizzle(raw) if swizzled else raw
    buf = torch.full((M, K + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.dequantize_fp4(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), swizzled, out=buf[:, :K])
    got = to_np(buf.double())
    want = plain.values_fp4(q, raw)
    assert np.array_equal(np.isnan(got[:, :K]), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[:, :K][ok], want[ok])
    assert np.array_equal(np.signbit(got[:, :K][ok]), np.signbit(want[ok]))
    assert np.all(got[:, K:] == 7.0)


# ---- products ----------------------------------------------------------------------------------------

def operand(M, K, seed, std=1.0, scale_spread=6):
    """(packed codes, raw scales, fp64 values) of random codes under scales of a few binades."""
    g = np.random.default_rng(seed)
    q = g.integers(0, 256, (M, K // 2), dtype=np.uint8)
    s = (127 + g.integers(-scale_spread, scale_spread + 1, (M, K // 32))).astype(np.uint8)
    return q, s, plain.values_fp4(q, s)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# K: one block, a half MMA, one MMA, one scale block, more than one (odd count), whole stages, a ragged last stage.
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 40, 64), (5, 256, 96), (128, 256, 128), (129, 257, 160), (256, 512, 256),
                                   (300, 200, 288), (64, 640, 384), (257, 130, 416), (16, 1000, 2048), (513, 300, 1056)])
def test_gemm(M, N, K, out_dtype):
    qa, sa, a = operand(M, K, M + K)
    qb, sb, b = operand(N, K, N + K + 1)
    c = mx.gemm_fp4(cuda(qa), cuda(oracle.swizzle(sa)), cuda(qb), cuda(oracle.swizzle(sb)), out_dtype=out_dtype)
    assert mx.device_error() == 0
    assert_gemm_close(to_np(c.float()), a @ b.T, np.abs(a) @ np.abs(b).T, out_dtype == torch.bfloat16, f"{M}x{N}x{K}")


# At most 64 rows: every token-tile width (16, 32, 64 and the first row count past them), K split over 1, 2, 4 and 8
# CTAs with equal and unequal shares, N that ends inside a tile.
@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 1024), (130, 2080), (260, 4128), (33, 6400)])
def test_gemm_few_rows(M, N, K):
    for out_dtype in (torch.float32, torch.bfloat16):
        test_gemm(M, N, K, out_dtype)


def test_gemm_few_rows_strided_output_and_nan_row():
    M, N, K = 40, 300, 4096
    qa, sa, a = operand(M, K, 11)
    qb, sb, b = operand(N, K, 12)
    sa[7, 100], sb[250, 3] = 255, 255
    buf = torch.full((M + 2, N + 5), 3.0, device="cuda")
    mx.gemm_fp4(cuda(qa), cuda(oracle.swizzle(sa)), cuda(qb), cuda(oracle.swizzle(sb)), out=buf[1:M + 1, :N])
    c = to_np(buf[1:M + 1, :N])
    bad = np.zeros((M, N), bool)
    bad[7], bad[:, 250] = True, True
    assert np.array_equal(np.isnan(c), bad)
    ok = ~bad
    assert_gemm_close(c[ok], (a @ b.T)[ok], (np.abs(a) @ np.abs(b).T)[ok], False, "beside NaN")
    assert torch.all(buf[:, N:] == 3.0) and torch.all(buf[0] == 3.0) and torch.all(buf[M + 1] == 3.0)


def test_gemm_many_tiles_per_pair_and_strided_output():
    """More tiles than CTA pairs (both accumulators in turn), and an output with untouched padding columns."""
    M, N, K = 2600, 2100, 512
    qa, sa, a = operand(M, K, 1)
    qb, sb, b = operand(N, K, 2)
    buf = torch.full((M, N + 9), 3.0, device="cuda")
    mx.gemm_fp4(cuda(qa), cuda(oracle.swizzle(sa)), cuda(qb), cuda(oracle.swizzle(sb)), out=buf[:, :N])
    assert_gemm_close(to_np(buf[:, :N]), a @ b.T, np.abs(a) @ np.abs(b).T, False, "strided")
    assert torch.all(buf[:, N:] == 3.0)


def test_nan_scale_of_one_row_stays_in_its_row():
    """A NaN block of A makes its row NaN and no other: neither rows of the same tile nor, K ending inside a scale
    block or with an odd count of them, the K-blocks that are not there."""
    for M, N, K in ((200, 128, 96), (200, 300, 128 * 3)):
        qa, sa, a = operand(M, K, 3)
        qb, sb, b = operand(N, K, 4)
        sa[130, 1] = 255
        c = to_np(mx.gemm_fp4(cuda(qa), cuda(oracle.swizzle(sa)), cuda(qb), cuda(oracle.swizzle(sb)), out_dtype=torch.float32))
        assert np.isnan(c[130]).all()
        keep = np.arange(M) != 130
        assert_gemm_close(c[keep], (a @ b.T)[keep], (np.abs(a) @ np.abs(b).T)[keep], False, "rows beside a NaN row")


def grouped(counts, N, K, out_dtype, seed, out=None):
    counts = [int(c) for c in counts]
    off = np.concatenate([[0], np.cumsum(counts)])
    G = len(counts)
    qa, sa, a = operand(int(off[-1]), K, seed)
    qb, sb, b = operand(G * N, K, seed + 1)
    swz_b = np.concatenate([oracle.swizzle(sb[g * N:(g + 1) * N]) for g in range(G)])
    c = mx.grouped_gemm_fp4(cuda(qa), cuda(oracle.swizzle(sa, counts)), cuda(qb.reshape(G, N, K // 2)), cuda(swz_b),
                            cuda(off.astype(np.int32)), out_dtype=out_dtype, out=out)
    ref, size = np.zeros((off[-1], N)), np.zeros((off[-1], N))
    for g in range(G):
        r = slice(off[g], off[g + 1])
        ref[r], size[r] = a[r] @ b[g * N:(g + 1) * N].T, np.abs(a[r]) @ np.abs(b[g * N:(g + 1) * N]).T
    assert mx.device_error() == 0
    assert_gemm_close(to_np(c.float()), ref, size, c.dtype == torch.bfloat16, f"grouped {counts} {N} {K}")


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(384, 256), (200, 32), (130, 160), (640, 384), (128, 896)])
def test_grouped(N, K, out_dtype):
    grouped([0, 5, 128, 129, 300, 0, 1, 64, 256, 257, 511, 2], N, K, out_dtype, K)


@pytest.mark.parametrize("counts", [[1], [0, 0, 3], [130, 0, 0], [0] * 70 + [40] + [0] * 57 + [3]])
def test_grouped_few_rows(counts):
    grouped(counts, 256, 128, torch.float32, 9)


# At most 32 rows per expert on average, with experts of 0, 1, 31, 32, 33, 127, 128, 129 and 300 rows among them.
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts", [[32, 0, 33, 1, 31, 0, 64, 0], [300] + [0] * 9, [0] * 6 + [127, 1], [128, 129] + [0] * 7, [5] * 40,
                                    [0] * 70 + [40] + [0] * 57 + [3], [32] * 3])
@pytest.mark.parametrize("N,K", [(128, 256), (130, 96), (384, 1056), (1, 32)])
def test_grouped_few_rows_per_expert(N, K, counts, out_dtype):
    grouped(counts, N, K, out_dtype, len(counts) + N)


def test_grouped_few_rows_many_tiles_and_strided_output():
    """More tiles than CTAs (the ring and the accumulator go round), and untouched columns beside the output."""
    g = np.random.default_rng(3)
    counts = g.integers(0, 40, 60)
    buf = torch.full((int(counts.sum()), 1400 + 3), 3.0, device="cuda")
    grouped(counts, 1400, 512, torch.float32, 5, out=buf[:, :1400])
    assert torch.all(buf[:, 1400:] == 3.0)


@pytest.mark.parametrize("rows", [128, 20])       # the pair kernel's grouped form and the one for few rows per expert
def test_grouped_bad_offsets_write_nothing(rows):
    h = rows // 2
    qa, sa, _ = operand(rows, 128, 1)
    qb, sb, _ = operand(512, 128, 2)
    out = torch.full((rows, 256), 3.0, device="cuda")
    mx.device_error()
    for bad in ([0, rows - 3, h], [0, h, rows - 1], [1, h, rows]):
        mx.grouped_gemm_fp4(cuda(qa), cuda(oracle.swizzle(sa, [h, h])), cuda(qb.reshape(2, 256, 64)), cuda(oracle.swizzle(sb)),
                            torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        assert mx.device_error() == 2
    assert torch.all(out == 3.0)


def test_expired_waits_end_the_grouped_product_for_few_rows_cleanly():
    G, N, K, rows = 8, 8192, 32768, 200
    g = torch.Generator(device="cuda").manual_seed(1)
    qa, qb = (torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda") for s in ((rows, K // 2), (G, N, K // 2)))
    sa = torch.full((mx.grouped_scale_bytes_bound(rows, G, K // 32),), 127, dtype=torch.uint8, device="cuda")
    sb = torch.full((G * mx.swizzled_scale_bytes(N, K // 32),), 127, dtype=torch.uint8, device="cuda")
    off = torch.arange(0, rows + 1, rows // G, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert mx.device_error() == 0
    mx.set_wait_timeout_ns(1)
    try:
        for _ in range(8):
            mx.grouped_gemm_fp4(qa, sa, qb, sb, off)
            torch.cuda.synchronize()
            bits = mx.device_error()
            if bits:
                break
    finally:
        mx.set_wait_timeout_ns(0)
    assert bits == 1
    grouped([5] * 40, 130, 96, torch.float32, 3)


def test_quantized_linear_all_three_products():
    """fprop, dgrad and wgrad of one linear layer from mx.quantize_fp4's own outputs (both directions), each against
    fp64 on the values its codes stand for."""
    M, N, K = 288, 352, 416
    X, W, dY = (synth.normal_bf16(s, seed=i) for i, s in enumerate(((M, K), (N, K), (M, N))))
    qx, qw, qd = (mx.quantize_fp4(t.cuda(), colwise=True) for t in (X, W, dY))

    def val(t):
        code, s = plain.quantize_fp4(t)
        return plain.values_fp4(plain.pack(code), s)

    x, w, d = f64(X), f64(W), f64(dY)
    for name, got, a, b in (("fprop", mx.gemm_fp4(qx[0], qx[1], qw[0], qw[1], torch.float32), x, w),
                            ("dgrad", mx.gemm_fp4(qd[0], qd[1], qw[2], qw[3], torch.float32), d, w.T.copy()),
                            ("wgrad", mx.gemm_fp4(qd[2], qd[3], qx[2], qx[3], torch.float32), d.T.copy(), x.T.copy())):
        va, vb = val(a), val(b)
        assert_gemm_close(to_np(got), va @ vb.T, np.abs(va) @ np.abs(vb).T, False, name)


def test_large_forward_sampled():
    """5200 x 24576 x 4096 (a forward gate_up projection): first, last and tile-edge rows and columns."""
    M, N, K = 5200, 24576, 4096
    X = synth.fwd_activations(M, K, device="cuda")
    W = synth.normal_bf16((N, K), std=0.02, seed=3, device="cuda")
    qx, sx, _, _ = mx.quantize_fp4(X)
    qw, sw, _, _ = mx.quantize_fp4(W)
    c = mx.gemm_fp4(qx, sx, qw, sw)
    rows = np.array([0, 127, 128, 255, 256, 2600, 5119, 5120, 5199])
    cols = np.array([0, 1, 127, 128, 255, 256, 12345, 24319, 24320, 24575])

    def val(t, idx):
        code, s = plain.quantize_fp4(f64(t[torch.from_numpy(idx).cuda()].cpu()))
        return plain.values_fp4(plain.pack(code), s)

    a, b = val(X, rows), val(W, cols)
    got = to_np(c[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()].float())
    assert_gemm_close(got, a @ b.T, np.abs(a) @ np.abs(b).T, True, "large forward")
    # The scale bytes of the sampled rows sit at their places of the layout.
    pos = scale_positions(M, K // 32)
    _, sb = plain.quantize_fp4(f64(X[torch.from_numpy(rows).cuda()].cpu()))
    assert np.array_equal(to_np(sx)[pos[rows]], sb)


@pytest.mark.parametrize("M,N,K", [(64, 40960, 32768), (4096, 4096, 16384)])
def test_expired_waits_end_the_product_cleanly(M, N, K):
    """With a 1 ns deadline waits that do not succeed at once expire: the kernel records error bit 1, drains and
    returns, and the next product is right. Both kernels. A wait's first try may itself block for a while (the
    hardware's suspend window), so the sizes are such that a CTA's work outlasts it: the few-row kernel must not split
    K over a cluster, which would leave each CTA a few microseconds."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q = [torch.randint(0, 256, (n, K // 2), generator=g, dtype=torch.uint8, device="cuda") for n in (M, N)]
    s, t = (torch.full((mx.swizzled_scale_bytes(n, K // 32),), 127, dtype=torch.uint8, device="cuda") for n in (M, N))
    torch.cuda.synchronize()
    assert mx.device_error() == 0
    mx.set_wait_timeout_ns(1)
    try:
        for _ in range(8):
            mx.gemm_fp4(q[0], s, q[1], t)
            torch.cuda.synchronize()
            bits = mx.device_error()
            if bits:
                break
    finally:
        mx.set_wait_timeout_ns(0)
    assert bits == 1
    test_gemm(257, 130, 416, torch.float32)
    test_gemm(16, 1000, 2048, torch.float32)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_output_rows_at_every_alignment(fmt, out_dtype):
    """Offsets and row strides that leave rows on every element boundary give the same values as aligned ones, and nothing
    beside them is written."""
    M, N, K = 140, 331, 160
    a, b = (synth.normal_bf16((r, K), seed=r).cuda() for r in (M, N))
    if fmt == "mxfp4":
        args, f = (*mx.quantize_fp4(a)[:2], *mx.quantize_fp4(b)[:2]), mx.gemm_fp4
    else:
        args, f = (*mx.quantize(a)[:2], *mx.quantize(b)[:2]), mx.gemm
    want = torch.empty((M, 352), dtype=out_dtype, device="cuda")[:, :N]
    f(*args, out=want)
    for n in (N, 320, 257, 65, 64, 1):
        if fmt == "mxfp4":
            part = (*args[:2], *mx.quantize_fp4(b[:n].contiguous())[:2])
        else:
            part = (*args[:2], *mx.quantize(b[:n].contiguous())[:2])
        for offset, ld in ((0, 331), (1, 331), (1, 332), (2, 333), (3, 334), (5, 336), (7, 335), (8, 352)):
            buf = torch.full((offset + M * ld + 8,), -7.0, dtype=out_dtype, device="cuda")
            f(*part, out=buf.as_strided((M, n), (ld, 1), offset))
            expect = torch.full_like(buf, -7.0)
            expect.as_strided((M, n), (ld, 1), offset).copy_(want[:, :n])
            assert torch.equal(buf, expect), (n, offset, ld)
