"""The router's choice where tokens that fp32 decides and tokens that need fp64 stand side by side."""
import numpy as np
import pytest
import torch

import plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu


# Groups that cut lanes: their keys go through shared memory. 100 / 10 and 60 / 20 cut them everywhere; 384 / 2, whose
# groups are twelve lanes each, no power of two, and 1000 / 8 as well; 7 / 7 is merged by shuffles.
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,topk_groups", [(100, 10, 3), (60, 20, 7), (384, 2, 1), (1000, 8, 3), (7, 7, 3)])
def test_near_and_clear_tokens_in_one_block(E, groups, topk_groups, group_score):
    """Every fourth, third or second token has keys nearer together than fp32 tells apart, its neighbours in the block have
    not, so a block's warps rank fp32 and fp64 keys at the same time. Each token's choice is what it is by itself.
    Weights: with u = 2^-24 and |x| < 12, (4 + 12) u for an exponential of each of numerator and sum, 2 u for 1 + e and its
    quotient on each side, k u for the sum, 2 u for the last quotient and product: under 50 u = 3e-6."""
    g = torch.Generator().manual_seed(E)
    near = 0.05 * torch.randn((1, E), generator=g)
    s = plain.scores(near[0].double().numpy(), "sigmoid")
    bias = torch.from_numpy(0.75 + 1e-9 * np.arange(E)[::-1] - s).float()
    near = near.repeat(16, 1)                       # the sigmoid's scores are independent: variants with experts off
    off = torch.rand((16, E), generator=g) < 0.2
    off[0] = False
    near[off] = float("-inf")
    clear = 2.0 * torch.randn((48, E), generator=g)
    rows = torch.cat([near, clear])
    k = min(6, E)
    args = dict(score="sigmoid", groups=groups, topk_groups=topk_groups, group_score=group_score)
    want, w64 = plain.route(rows.double().numpy(), k, bias=bias.double().numpy(), **args)
    T = 16000
    for every in (4, 3, 2):
        pick = torch.randint(16, 64, (T,), generator=g)
        pick[::every] = torch.randint(0, 16, (len(pick[::every]),), generator=g)
        x, at = rows[pick].cuda(), pick.numpy()
        for _ in range(5):
            ids, w = mx.route(x, k, bias=bias.cuda(), **args)
            assert np.array_equal(to_np(ids), want[at])
            assert np.allclose(to_np(w), w64[at], rtol=3e-6, atol=0)


def choice(x, k, **args):
    ids, _ = mx.route(x.cuda(), k, **{n: v.cuda() if torch.is_tensor(v) else v for n, v in args.items()})
    want, _ = plain.route(x.double().numpy(), k, **{n: v.double().numpy() if torch.is_tensor(v) else v for n, v in args.items()})
    assert np.array_equal(to_np(ids), want), (args, k, np.argwhere(to_np(ids) != want)[0])
    return to_np(ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_twins_at_the_border_hide_no_better_expert(dtype):
    """The last chosen expert and the best one left out have the same logit and bias; an expert behind them, whose fp32 key
    is no larger, has the larger fp64 key."""
    zero, same = torch.zeros(8), torch.full((8,), 3000.0)
    x = torch.tensor([[20.0, 20, 25, 0, 0, 0, 0, 0], [20, 20, 20.125, -5, -5, -5, -5, -5], [0, 20, 20, 20, 20, 20, 20, 25],
                      [30, 20, 20, 20, 21, 20, 24, 0]]).to(dtype)
    assert choice(x, 1, score="sigmoid", bias=zero)[:, 0].tolist() == [2, 2, 7, 0]
    for k in (2, 3, 4, 7):
        choice(x, k, score="sigmoid", bias=zero)
        choice(x, k, score="sigmoid", bias=same)
        choice(x, k, score="sigmoid", groups=2, topk_groups=1, group_score="top2")
        choice(x, k, score="sigmoid", groups=4, topk_groups=3, group_score="top2")
    y = torch.tensor([[0.0, -200, -200, -190, -300, -400, -410, -420], [0, -30, -30, -20, -40, -40, -30, -19.5],
                      [-30, -30, -30, -29, 0, -30, -28, -30]]).to(dtype)
    assert choice(y[:1], 2, bias=zero).tolist() == [[0, 3]]
    for k in range(1, 8):
        for bias in (zero, same, torch.full((8,), 0.25)):
            choice(y, k, bias=bias)
        choice(y, k, groups=2, topk_groups=1, group_score="top2")


@pytest.mark.parametrize("E,groups,topk_groups", [(8, 1, 1), (32, 1, 1), (60, 1, 1), (64, 8, 5), (100, 10, 6), (256, 1, 1), (1024, 4, 3)])
@pytest.mark.parametrize("score,low,high", [("sigmoid", 17, 36), ("softmax", -60, -17)])
def test_few_distinct_logits_whose_scores_fp32_merges(E, groups, topk_groups, score, low, high):
    """BF16 logits drawn from a few values where fp32 scores saturate or vanish, under constant biases: equal experts and
    hidden ones at every place of the order."""
    g = torch.Generator().manual_seed(E)
    for few in (2, 3, 6):
        T = 120 if E < 256 else 30
        values = (low + (high - low) * torch.rand((T, few), generator=g)).to(torch.bfloat16)
        x = torch.gather(values, 1, torch.randint(0, few, (T, E), generator=g))
        if score == "softmax":
            x[torch.arange(T), torch.randint(0, E, (T,), generator=g)] = 0.0
        for k in (1, 2, 5, 8):
            for b in (0.0, 0.25, 1000.0):
                choice(x, k, score=score, bias=torch.full((E,), b), groups=groups, topk_groups=topk_groups, group_score="max")
            choice(x, k, score=score, groups=groups, topk_groups=topk_groups, group_score="top2")


def test_equal_logits_everywhere():
    """All experts alike, as before the first update: the first k."""
    for E, k in ((128, 8), (100, 6)):
        x = torch.zeros((50, E))
        for score in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(E), torch.full((E,), 0.1)):
                assert (choice(x, k, score=score, bias=bias) == np.arange(k)).all()


def test_several_tokens_per_warp_where_they_begin():
    """BF16 logits that decide by themselves, at most 128 experts: 4 tokens per warp from 8192 on (k <= 8), 2 from 4096 on
    (k > 8), batches on both sides of each and with every tail. The same choice and weights as of the tokens by themselves."""
    g = torch.Generator().manual_seed(3)
    for E, k, sizes in ((128, 8, (8190, 8191, 8192, 8193, 8195)), (40, 3, (8191, 8194)), (17, 1, (8193,)), (64, 9, (4095, 4096, 4097)),
                        (128, 16, (4097,))):
        x = (4 * torch.randn((max(sizes), E), generator=g)).round() / 2
        x[torch.rand(x.shape, generator=g) < 0.2] = float("-inf")
        x[3] = float("-inf")
        x = x.to(torch.bfloat16).cuda()
        want = torch.sort(x.double(), dim=1, descending=True, stable=True)
        expect = torch.where(want.values[:, :k] > -np.inf, want.indices[:, :k], -1)
        groups = 8 if E % 8 == 0 else 1
        for renormalize in (True, False):
            parts = [mx.route(p, k, renormalize=renormalize) for p in x.split(1000)]
            of_groups = torch.cat([mx.route(p, k, groups=groups, topk_groups=max(1, groups // 2))[0] for p in x.split(1000)])
            ids1, w1 = (torch.cat(v) for v in zip(*parts))
            for T in sizes:
                ids, w = mx.route(x[:T], k, renormalize=renormalize)
                assert torch.equal(ids.long(), expect[:T]) and torch.equal(ids, ids1[:T]) and torch.equal(w, w1[:T])
                assert torch.equal(mx.route(x[:T], k, groups=groups, topk_groups=max(1, groups // 2))[0], of_groups[:T])
