"""GPU parity of the rotation table, rotary positions and their gradient.

Tolerances: a table entry is a fp64 value (error far below) rounded once, 2^-24 of it, and the test's own fp64 angle may differ in
its last bit: position * 2^-52. A rotated element is a sum of two products within 1.5 ulp of fp32 (3 * 2^-24 of it), rounded once:
half a step of the output type, relative to the value, and half the smallest subnormal of FP16."""
import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def near(got, want, dtype):
    got = got.double().cpu().numpy()
    bound = (HALF[dtype] + 3 * 2.0 ** -24) * np.abs(want) + TINY[dtype]
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / bound)


def tensor(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("rot,base,scaling,first", [(2, 10000.0, None, 0), (64, 500.0, ("linear", 4), 7), (128, 1e6, ("ntk", 8), 0),
                                                    (128, 1e4, ("yarn", 4, 4096), 100000), (256, 1e6, None, 1 << 20)])
def test_table(rot, base, scaling, first):
    freq, amplitude = mx.rope_frequencies(rot, base, scaling)
    got = to_np(mx.rope_table(301, rot, base, scaling, first=first)).astype(np.float64)
    a = (first + np.arange(301.0))[:, None] * np.array(freq)
    want = amplitude * np.concatenate([np.cos(a), np.sin(a)], 1)
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + amplitude * (first + 301) * 2.0 ** -51).all()


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (1, 32, 128, 128), (13, 5, 64, 32), (7, 3, 80, 16), (33, 8, 96, 96), (5, 2, 30, 14),
                                       (3, 1, 257, 256), (300, 9, 128, 64), (2, 40, 8, 6)])
def test_rope(T, H, D, rot, dtype, interleaved, back):
    x = tensor((T, H, D), dtype, T + D)
    tab = plain.table(500, plain.frequencies(rot))
    pos = np.random.default_rng(T).integers(0, 500, T)
    f = mx.rope_backward if back else mx.rope
    want = plain.rope(x.double().numpy(), tab, pos, interleaved, back)
    for kind in (torch.int32, torch.int64):
        got = f(x.cuda(), torch.from_numpy(tab).cuda(), torch.from_numpy(pos).to(kind).cuda(), interleaved)
        near(got, want, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_offsets_and_in_place(dtype, interleaved):
    """Views of a fused projection, rows that begin off 16 bytes, transposed heads, rotation in place."""
    T, H, D, rot = 37, 6, 64, 32
    tab = plain.table(64, plain.frequencies(rot))
    tab_d = torch.from_numpy(tab).cuda()
    flat = tensor((T * (H + 2) * D + 16,), dtype, 1)
    for start, make in ((0, lambda f: f[:T * (H + 2) * D].view(T, H + 2, D)[:, 1:H + 1]),
                        (1, lambda f: f[1:1 + T * H * D].view(T, H, D)),
                        (0, lambda f: f[:T * H * D].view(H, T, D).transpose(0, 1)),
                        (0, lambda f: f[:T * H * (D + 1)].view(T, H, D + 1)[:, :, :D] if T * H * (D + 1) <= f.numel() else f[:T * H * D].view(T, H, D))):
        x = make(flat)
        want = plain.rope(x.double().numpy(), tab, np.arange(T), interleaved)
        d = flat.cuda()
        xd = make(d)
        near(mx.rope(xd, tab_d, interleaved=interleaved), want, dtype)
        assert torch.equal(d.cpu(), flat)
        out = make(torch.zeros_like(d))
        assert mx.rope(xd, tab_d, interleaved=interleaved, out=out) is out
        near(out, want, dtype)
        rest = flat.cuda()
        make(rest).zero_()
        mx.rope(xd, tab_d, interleaved=interleaved, out=xd)          # in place: only the view changes
        near(xd, want, dtype)
        xd.zero_()
        assert torch.equal(d, rest)


def test_padding_and_positions_behind_the_table():
    x = tensor((5, 3, 64), torch.bfloat16, 3)
    tab = plain.table(10, plain.frequencies(32))
    pos = np.array([0, -1, 9, 10, 1 << 40])
    mx.device_error()
    got = mx.rope(x.cuda(), torch.from_numpy(tab).cuda(), torch.from_numpy(pos).cuda())
    near(got, plain.rope(x.double().numpy(), tab, pos, False), torch.bfloat16)
    assert mx.device_error() == 4
    mx.rope(x.cuda(), torch.from_numpy(tab).cuda(), torch.from_numpy(np.minimum(pos, 9)).cuda())
    assert mx.device_error() == 0                                   # a negative position is padding, no error


def test_cancellation_and_infinities():
    """Where the two products cancel the result keeps its relative accuracy; infinite inputs stay infinite."""
    tab = torch.tensor([[0.75, 0.75], [1.0, 0.5]], device="cuda")
    x = torch.tensor([[[1.0, 1.0 - 2.0 ** -24]], [[float("inf"), 3.0]]], device="cuda")
    y = mx.rope(x, tab)
    assert y[0, 0, 0].item() == 0.75 * 2.0 ** -24
    assert y[1, 0, 0].item() == float("inf") and y[1, 0, 1].item() == float("inf")


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_formulas_and_the_differences(interleaved):
    """<dx, v> equals <dy, rope(x + h v) - rope(x - h v)> / 2 h: the map is linear, so h = 1 and only roundings are left."""
    T, H, D, rot = 6, 3, 32, 24
    tab = torch.from_numpy(plain.table(50, plain.frequencies(rot), 1.3)).cuda()
    pos = torch.tensor([0, 3, 49, 7, 7, 20], dtype=torch.int32, device="cuda")
    x, v, dy = (tensor((T, H, D), torch.float32, i).cuda() for i in range(3))
    dx = mx.rope_backward(dy, tab, pos, interleaved)
    diff = (mx.rope(x + v, tab, pos, interleaved).double() - mx.rope(x - v, tab, pos, interleaved).double()) / 2
    a, b = (dx.double() * v.double()).sum(), (dy.double() * diff).sum()
    n = (dy.double().abs() * (x.abs() + v.abs()).double()).sum() * 2.6
    assert abs(a - b) <= n * 8 * 2.0 ** -24
    leaf = x.double().cpu().requires_grad_(True)
    near(dx, plain.rope(dy.double().cpu().numpy(), tab.cpu().numpy(), pos.cpu().numpy(), interleaved, back=True), torch.float32)
    assert leaf.grad is None


def test_captured_and_on_another_stream():
    x = tensor((9, 4, 128), torch.bfloat16, 5).cuda()
    tab = mx.rope_table(64, 128)
    want = mx.rope(x, tab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(mx.rope(x, tab), want)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mx.rope(x, tab)
        back = mx.rope_backward(y, tab)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, mx.rope(x, tab)) and torch.equal(back, mx.rope_backward(y, tab))
