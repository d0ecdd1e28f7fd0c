"""Waits that run out: the kernel records its error bit, drains and returns, and later calls are right."""
import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx
from test_gpu_fp4 import grouped, test_gemm as check_gemm

pytestmark = pytest.mark.gpu


def expire(call, tries=8):
    """Calls under a 1 ns deadline until a wait has run out; the error bits."""
    torch.cuda.synchronize()
    assert mx.device_error() == 0
    mx.set_wait_timeout_ns(1)
    try:
        for _ in range(tries):
            call()
            torch.cuda.synchronize()
            bits = mx.device_error()
            if bits:
                break
    finally:
        mx.set_wait_timeout_ns(0)
    return bits


def codes(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device="cuda")


def ones(n):
    return torch.full((n,), 127, dtype=torch.uint8, device="cuda")


def test_mxfp4_grouped_pair_kernel():
    G, N, K, rows = 4, 4096, 16384, 2048
    off = torch.arange(0, rows + 1, rows // G, dtype=torch.int32, device="cuda")
    args = (codes(1, rows, K // 2), ones(mx.grouped_scale_bytes_bound(rows, G, K // 32)), codes(2, G, N, K // 2),
            ones(G * mx.swizzled_scale_bytes(N, K // 32)), off)
    for _ in range(3):
        assert expire(lambda: mx.grouped_gemm_fp4(*args)) == 1
        grouped([300, 0, 129, 70], 130, 416, torch.float32, 3)
        check_gemm(257, 130, 416, torch.float32)


# K in one piece, over 2, and over 8 CTAs of a cluster. Sizes as in the library's other tests of expired waits: a CTA's work has
# to outlast a wait's first try.
@pytest.mark.parametrize("M,N,K", [(64, 40960, 32768), (64, 18816, 65536), (16, 2048, 524288)])
def test_few_rows_write_no_sums_of_unfinished_parts(M, N, K):
    """After an expired wait every element of the output is the product's or untouched, whichever CTAs gave up."""
    args = (codes(1, M, K // 2), ones(mx.swizzled_scale_bytes(M, K // 32)), codes(2, N, K // 2), ones(mx.swizzled_scale_bytes(N, K // 32)))
    want = mx.gemm_fp4(*args, out_dtype=torch.float32)
    assert mx.device_error() == 0
    expired = 0
    try:
        for ns in (1, 1, 3000, 10000, 20000, 30000, 50000, 70000, 90000, 120000) * 3:
            out = torch.full_like(want, -7.0)
            mx.set_wait_timeout_ns(ns)
            mx.gemm_fp4(*args, out=out)
            torch.cuda.synchronize()
            bits = mx.device_error()
            assert bits in (0, 1)
            expired += bits
            mixed = (out != want) & (out != -7.0)
            assert not mixed.any(), f"{int(mixed.sum())} elements after {ns} ns"
            if not bits:
                assert torch.equal(out, want)
    finally:
        mx.set_wait_timeout_ns(0)
    assert expired > 0
    assert torch.equal(mx.gemm_fp4(*args, out_dtype=torch.float32), want)
