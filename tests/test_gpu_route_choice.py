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
