"""The compiled call path: output sizes against the library's own arithmetic, and arguments that are no arguments."""
import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 32), (1, 8, 128, 64), (13, 8, 128, 2048), (127, 1, 3, 96), (128, 1, 1, 160), (129, 2, 700, 32),
                                     (300, 4, 16, 4096), (5, 3, 1024, 416)])
def test_output_sizes(T, k, E, K):
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k)
    off, slot_row, counts = mx.route_plan(ids, E)
    assert off.shape == (E + 1,) and slot_row.shape == ids.shape and counts.shape == (E,)
    for fmt, width in (("mxfp8", K), ("mxfp4", K // 2)):
        q, s = mx.dispatch_quantize(x, slot_row, off, fmt)
        assert q.shape == (T * k, width) and s.numel() == mx.grouped_scale_bytes_bound(T * k, E, K // 32)
    q, s, _, _ = mx.quantize_fp4(x)
    assert q.shape == (T, K // 2) and s.numel() == mx.swizzled_scale_bytes(T, K // 32)
    assert mx.dequantize_fp4(q, s).shape == (T, K)
    if T % 32 == 0:
        _, _, q, s = mx.quantize_fp4(x, rowwise=False, colwise=True)
        assert q.shape == (K, T // 2) and s.numel() == mx.swizzled_scale_bytes(K, T // 32)


def test_python_errors_come_through():
    x = torch.zeros((4, 8), device="cuda")
    for bad in (2.5, "2", None):
        with pytest.raises(TypeError):
            mx.route(x, bad)
    with pytest.raises(TypeError):
        mx.route(x, 2, scale="much")
    with pytest.raises(OverflowError):
        mx.route_plan(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 1 << 70)
    with pytest.raises(mx.MxError):
        mx.route(x, 2, out=(torch.empty((4, 2), device="cuda"),) * 2)      # ids are int32
    with pytest.raises(mx.MxError):
        mx.route_plan(torch.zeros((4, 2), dtype=torch.int64, device="cuda"), 4)
    ids, w = mx.route(x, torch.tensor(2))                                   # anything with __index__
    assert ids.shape == (4, 2)


def test_rows_that_no_slot_names_get_a_zero_gradient():
    """More or fewer rows than slots: what no slot names is 0 in the gradient that the binding allocates."""
    slot_row = torch.tensor([[0, 5], [-2 ** 31, 2], [7, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    for rows in (5, 8, 11):
        c, dy = torch.randn((rows, 40), device="cuda"), torch.ones((3, 40), device="cuda")
        junk = torch.full((rows, 40), 9.0, device="cuda")
        del junk                                                            # what a new tensor of that size may hold
        d, _ = mx.combine_backward(dy, c, slot_row)
        want = torch.zeros((rows, 40), device="cuda")
        want[[r for r in (0, 2, 5, 7) if r < rows]] = 1.0
        assert torch.equal(d, want)
