"""GPU parity of the router: the choice exactly, weights and gradients within fp32 rounding of fp64.

Tolerances (u = 2^-24, half an fp32 step): CUDA's expf is off by at most 2 ulp = 4 u; its argument x - m by u |x - m|,
which the exponential carries over as a relative error; a sum of n terms by n u; a product or a division by u. With
D = the largest |x - m| that matters and n <= E terms, one weight is off by at most (2 (4 + D) + n + 4) u relative,
numerator and denominator together; sigmoid's 1 / (1 + e) adds 2 u. A gradient multiplies three such factors."""
import numpy as np
import pytest
import torch

import plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def logits(T, E, seed, dtype, masked=False, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn((T, E), generator=g)
    if masked:
        x[:, torch.rand(E, generator=g) < 0.3] = float("-inf")
        x[T // 2] = float("-inf")
        x[T - 1, 1:] = float("nan")
    return x.to(dtype)


def relative(E, x):
    x = plain.clean(x)
    live = x > -np.inf
    D = 0.0
    for t in range(len(x)):
        if live[t].any():
            D = max(D, min(104.0, x[t][live[t]].max() - x[t][live[t]].min()))     # past 104 fp32's e^-d is 0
    return (2 * (4 + D) + E + 8) * U


def check(x, k, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renormalize=True, scale=1.0, seed=0,
          backward=True):
    T, E = x.shape
    dx = x.cuda()
    args = dict(score=score, renormalize=renormalize, scale=scale)
    more = dict(bias=None if bias is None else bias.cuda(), groups=groups, topk_groups=topk_groups, group_score=group_score)
    ids, w = mx.route(dx, k, **args, **more)
    x64 = x.double().numpy()
    more["bias"] = None if bias is None else bias.double().numpy()
    want, w64 = plain.route(x64, k, **args, **more)
    assert np.array_equal(to_np(ids), want)
    rel = relative(E, x64)
    err = np.abs(to_np(w) - w64)
    assert np.all(err <= rel * np.abs(w64) + abs(scale) * 2.0 ** -126), f"weights {err.max()}"
    if not backward:
        return ids, w
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(seed + 7))
    d = mx.route_backward(dw.cuda(), dx, ids, **args)
    assert d.dtype == x.dtype
    d64, size = plain.route_backward(dw.double().numpy(), x64, want, **args)
    bound = (3 * rel + (k + 8) * U) * size + HALF[x.dtype] * np.abs(d64) + 2.0 ** -120
    assert np.all(np.abs(to_np(d.double()) - d64) <= bound), "gradient"
    return ids, w


# E: one lane's worth, fewer than a warp, whole and ragged multiples of every vector width, the largest.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 8), (33, 31, 4), (17, 32, 1), (40, 60, 6), (64, 100, 8), (130, 128, 8),
                                   (50, 160, 6), (70, 256, 8), (9, 384, 16), (6, 513, 10), (5, 1000, 9), (4, 1024, 16)])
def test_sizes(T, E, k, score, dtype):
    check(logits(T, E, E + k, dtype), k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("masked", [True, False])
def test_forms(score, renormalize, biased, masked):
    x = logits(120, 96, 3, torch.float32, masked)
    b = 0.1 * torch.randn(96, generator=torch.Generator().manual_seed(1)) if biased else None
    check(x, 6, score, b, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,topk_groups", [(256, 8, 4), (100, 10, 3), (96, 32, 5), (64, 4, 4), (60, 20, 1), (32, 32, 8), (7, 7, 3)])
@pytest.mark.parametrize("biased", [True, False])
def test_groups(E, groups, topk_groups, group_score, score, biased):
    """Groups inside lanes, across lanes and of one expert; with masked experts some groups hold none or one."""
    x = logits(90, E, E + groups, torch.float32, masked=True)
    b = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(2)) if biased else None
    check(x, min(5, E), score, b, groups, topk_groups, group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score):
    """BF16 logits on a coarse grid: equal logits (and equal or zero biases) everywhere."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randint(-3, 4, (300, 128), generator=g) / 2).to(torch.bfloat16)
    for b in (None, torch.zeros(128), (torch.randint(0, 3, (128,), generator=g) / 64).float()):
        check(x, 8, score, b, 8, 3, "top2", backward=False)
        check(x, 8, score, b, backward=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_nearer_than_fp32_tells_apart(score):
    """Biases built so that score + bias of many experts differ by 1e-9 or less: the choice is the fp64 one."""
    E, T = 64, 40
    g = torch.Generator().manual_seed(5)
    x = 0.05 * torch.randn((T, E), generator=g)
    row = x[0].double().numpy()
    target = 0.75 + 1e-9 * np.arange(E)[::-1]
    b = torch.from_numpy(target - plain.scores(row, score)).float()
    check(x, 8, score, b, backward=False)
    check(x, 8, score, b, 8, 2, "top2", backward=False)
    check(x[:1].repeat(T, 1), 8, score, b, 16, 5, "max", backward=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_extreme_logits(score, renormalize):
    """Far negative (sigmoid underflows), far positive, the type's lowest value as a mask, infinities, one expert left."""
    rows = [[-200.0, -201.0, -200.5, -500.0], [300.0, 299.0, -300.0, 0.0], [-3.0e38, -3.0e38, 1.0, -3.0e38],
            [-3.3e38] * 4, [float("inf"), 1.0, float("inf"), 0.0], [float("-inf")] * 3 + [-1000.0],
            [float("nan"), float("-inf"), float("-inf"), float("nan")], [-59.0, -60.5, -61.0, -90.0], [-60.5, -61.0, -62.0, -99.0]]
    check(torch.tensor(rows), 3, score, renormalize=renormalize)
    check(torch.tensor(rows), 4, score, renormalize=renormalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_extreme_logits_with_bias_and_groups(score, group_score):
    """The same range of logits where scores and biases are added: saturated and vanishing scores, equal keys."""
    rows = torch.tensor([[-200.0, -201.0, 300.0, 299.0, 0.0, -3.0e38, 1.0, 40.0], [50.0, 60.0, 70.0, 80.0, 90.0, 100.0, 45.0, 44.0],
                         [-3.3e38] * 8, [float("inf"), 1.0, float("inf"), 0.0, float("-inf"), float("nan"), 2.0, 2.0],
                         [float("-inf")] * 7 + [-1000.0], [-300.0, -310.0, -320.0, -330.0, -340.0, -350.0, -360.0, -370.0]])
    for b in (torch.zeros(8), torch.full((8,), 0.25), torch.linspace(-1, 1, 8), torch.linspace(1e4, 2e4, 8)):
        check(rows, 5, score, b, backward=False)
        check(rows, 3, score, b, 4, 2, group_score, backward=False)
        check(rows.to(torch.bfloat16), 4, score, b, 2, 1, group_score, backward=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(score):
    """Groups whose two largest keys nearly cancel: the sums differ by far less than a key's fp32 rounding."""
    E, T, B = 32, 30, 3000.0
    x = logits(T, E, 3, torch.float32, spread=0.5)
    b = torch.full((E,), -9.0e4)
    g = torch.Generator().manual_seed(1)
    for i in range(8):
        b[4 * i], b[4 * i + 2] = B * (i + 1), -B * (i + 1) + 1e-3 * torch.rand((), generator=g)
    check(x, 6, score, b, 8, 3, "top2", backward=False)
    check(x, 2, score, b / 1000, 8, 1, "top2", backward=False)


def test_bias_that_cannot_be_chosen():
    x = logits(20, 16, 1, torch.float32)
    b = torch.zeros(16)
    b[3], b[5], b[9] = float("-inf"), float("nan"), float("inf")
    ids, _ = check(x, 16, "sigmoid", b)
    got = to_np(ids)
    assert not np.isin(got, [3, 5]).any() and np.all(got[:, 0] == 9) and np.all(got[:, 14:] == -1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_offsets_and_outputs(dtype):
    """Rows that no vector load can take, and outputs with untouched neighbours."""
    T, E, k = 37, 64, 4
    for pad, off in ((1, 0), (8, 0), (0, 1), (3, 1)):
        flat = torch.randn(T * (E + pad) + off, generator=torch.Generator().manual_seed(pad)).to(dtype).cuda()
        x = flat[off:].view(T, E + pad)[:, :E]
        ids, w = mx.route(x, k)
        ids2, w2 = mx.route(x.contiguous(), k)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
        buf = torch.full((T, E + 5), 9.0, dtype=dtype, device="cuda")
        dw = torch.randn((T, k), device="cuda")
        for renorm in (True, False):
            mx.route_backward(dw, x, ids, renormalize=renorm, out=buf[:, :E])
            assert torch.equal(buf[:, :E], mx.route_backward(dw, x.contiguous(), ids, renormalize=renorm))
            assert torch.all(buf[:, E:] == 9.0)


def test_backward_skips_ids_outside_and_adds_repeated_ones():
    x = logits(6, 10, 2, torch.float32)
    ids = np.array([[1, -1, 3], [10, 2, 2], [-7, -1, -1], [0, 9, 0], [4, 5, 6], [1 << 30, 0, 1]])
    dw = torch.randn((6, 3), generator=torch.Generator().manual_seed(3))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = mx.route_backward(dw.cuda(), x.cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(), score, renorm)
            d64, size = plain.route_backward(dw.double().numpy(), x.double().numpy(), ids, score, renorm)
            rel = relative(10, x.double().numpy())
            assert np.all(np.abs(to_np(d.double()) - d64) <= (3 * rel + 16 * U) * size + U * np.abs(d64) + 2.0 ** -120)


def test_large_batch_against_torch_sort():
    """20 480 tokens of 128 experts: every choice against a stable sort in fp64 on the device."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((20480, 128), generator=g, device="cuda")
    b = 0.05 * torch.randn(128, generator=g, device="cuda")
    for score in ("softmax", "sigmoid"):
        s = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
        want = torch.sort(s + b.double(), dim=1, descending=True, stable=True).indices[:, :8]
        ids, w = mx.route(x, 8, score, b)
        assert torch.equal(ids.long(), want)
        chosen = torch.gather(s, 1, want)
        assert torch.allclose(w.double(), chosen / chosen.sum(1, keepdim=True), rtol=relative(128, x[:64].cpu().double().numpy()), atol=0)


def test_empty_batch():
    x = torch.empty((0, 8), device="cuda")
    ids, w = mx.route(x, 2)
    assert ids.shape == (0, 2) and mx.route_backward(w, x, ids).shape == (0, 8)


# ---- the row partition -------------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (13, 8, 128), (512, 8, 7), (513, 8, 64), (5000, 1, 1000), (5000, 3, 1024),
                                   (1024, 8, 33), (2049, 4, 1024), (4096, 8, 16), (4097, 8, 128), (32769, 1, 5), (20480, 8, 128), (300000, 2, 60)])
@pytest.mark.parametrize("dropped", [False, True])
def test_plan(T, k, E, dropped):
    g = np.random.default_rng(T + E)
    ids = np.minimum((E * g.random((T, k)) ** 2).astype(np.int64), E - 1)       # uneven loads
    if dropped:
        ids[g.random((T, k)) < 0.2] = -1
        ids[0, 0], ids[-1, -1] = E, -2 ** 31
    off, slot_row, counts = mx.route_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    o, s, c = plain.plan(ids, E)
    assert np.array_equal(to_np(off), o) and np.array_equal(to_np(counts), c) and np.array_equal(to_np(slot_row), s)


@pytest.mark.parametrize("T", [3000, 9000])
def test_plan_in_a_graph_and_two_at_once(T):
    """A cluster's sort, and two kernels, the second launched early: captured and replayed on other ids, and two calls
    on two streams at the same time, each with its own workspace."""
    k, E = 8, 100
    g = np.random.default_rng(8)
    draw = lambda: torch.from_numpy(g.integers(-1, E, (T, k)).astype(np.int32))  # noqa: E731
    ids = draw().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.route_plan(ids, E)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.route_plan(ids, E)
    for _ in range(3):
        new = draw()
        ids.copy_(new)
        graph.replay()
        for got, want in zip(out, plain.plan(new.numpy(), E)):
            assert np.array_equal(to_np(got), want)
    a, b = draw().cuda(), draw().cuda()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    res = []
    for _ in range(5):
        with torch.cuda.stream(side):
            res.append((a, mx.route_plan(a, E)))
        with torch.cuda.stream(other):
            res.append((b, mx.route_plan(b, E)))
    torch.cuda.synchronize()
    for x, out in res:
        for got, want in zip(out, plain.plan(to_np(x), E)):
            assert np.array_equal(to_np(got), want)


def test_many_tokens_per_warp_with_every_tail():
    """Batches above the size where a warp takes several tokens, ending inside a warp's tokens."""
    for T, E, k in ((4096, 40, 8), (4097, 128, 3), (4099, 64, 16), (5003, 17, 9), (4098, 128, 8)):
        x = logits(T, E, T + k, torch.bfloat16, masked=True)
        x[::7] = (x[::7] * 2).round() / 2                             # ties
        x[5, :2] = torch.tensor([float("inf"), 3.38e38])
        want = torch.sort(torch.nan_to_num(x.double(), nan=float("-inf"), posinf=3.4028234e38, neginf=float("-inf")), dim=1, descending=True, stable=True)
        for renorm in (True, False):
            ids, w = mx.route(x.cuda(), k, renormalize=renorm)
            exp = torch.where(want.values[:, :k] > -np.inf, want.indices[:, :k], -1)
            assert torch.equal(ids.cpu().long(), exp)
            sub = slice(0, 200)
            _, w64 = plain.route(x[sub].double().numpy(), k, renormalize=renorm)
            assert np.all(np.abs(to_np(w)[sub] - w64) <= relative(E, x[sub].double().numpy()) * w64 + 2.0 ** -126)


def test_plan_without_slots_and_without_experts():
    off, slot_row, counts = mx.route_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 5)
    assert to_np(off).tolist() == [0] * 6 and to_np(counts).tolist() == [0] * 5 and slot_row.shape == (0, 4)
    off, slot_row, counts = mx.route_plan(torch.full((9000,), -1, dtype=torch.int32, device="cuda"), 5)
    assert to_np(off).tolist() == [0] * 5 + [9000] and not to_np(counts).any()
    assert np.array_equal(to_np(slot_row), ~np.arange(9000))
