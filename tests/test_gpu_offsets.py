"""Row offsets that are no partition: every grouped product reports them and writes nothing."""
import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu

# Differences of neighbours that wrap in 32 bits to numbers >= 0 whose sum comes back to the row count, and some that do not.
WRAPPED = [[0, 2 ** 30, -2 ** 31, -2 ** 30, 0], [0, 2 ** 31 - 1, -2, 0, 0], [0, 1, 2 ** 31 - 1, -2 ** 31 + 5, 7],
           [0, -1, 3, 5, 9], [0, -2 ** 31, 0, 4, 5]]


def operands(rows, G, N, K, fp4):
    g = torch.Generator(device="cuda").manual_seed(rows)
    u8 = lambda *s: torch.randint(0, 100, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    one = lambda n: torch.full((n,), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    w = K // 2 if fp4 else K
    return (u8(rows, w), one(mx.grouped_scale_bytes_bound(rows, G, K // 32)), u8(G, N, w),
            one(G * mx.swizzled_scale_bytes(N, K // 32)))


@pytest.mark.parametrize("bad", WRAPPED)
@pytest.mark.parametrize("kind", ["mxfp8 pair", "mxfp8 single", "swiglu", "mxfp4", "mxfp4 few"])
def test_offsets_that_wrap(kind, bad):
    rows, N, K, G = (20 if kind == "mxfp4 few" else 320), 256, 128, 5
    args = operands(rows, G, N, K, "mxfp4" in kind)
    off = torch.tensor(bad + [rows], dtype=torch.int32, device="cuda")
    assert mx.device_error() == 0
    if kind == "swiglu":
        h = torch.full((rows, N // 2), 3, dtype=torch.uint8, device="cuda")
        s = torch.full((mx.grouped_scale_bytes_bound(rows, G, N // 64),), 3, dtype=torch.uint8, device="cuda")
        mx.grouped_gemm_swiglu_quant(*args, off, None, out=(h, s))
        outs = (h, s)
    else:
        outs = (torch.full((rows, N), 3.0, device="cuda"),)
        mx.set_gemm_variant(1 if kind == "mxfp8 single" else 0)
        try:
            (mx.grouped_gemm_fp4 if "mxfp4" in kind else mx.grouped_gemm)(*args, off, out=outs[0])
        finally:
            mx.set_gemm_variant(0)
    assert mx.device_error() == 2
    assert all(torch.all(o == 3) for o in outs)
