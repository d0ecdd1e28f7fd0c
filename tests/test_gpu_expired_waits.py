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
