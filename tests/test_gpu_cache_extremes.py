"""Attention at the ends of what its arguments may be: as many tokens as an int32 counts, scores as large as fp32 tells apart."""
import math

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32

pytestmark = pytest.mark.gpu


def test_a_sequence_of_all_the_tokens_an_int32_counts():
    """2^31 - 1 keys with one score, in pages that the table names again and again. Nothing stands in the last page's last place, whose
    zero codes would outweigh all: scores are -300. Sums: a lane adds fewer than 2^17 terms, 2^-7 relative; tensor-core sums of as
    many steps truncate, 2^-6."""
    D, page, pages = 64, 128, 1024
    cache = mx.cache_create(pages, 1, D, page)
    cache.k.fill_(0xB8)                                             # -1
    cache.v.fill_(0x40)                                             # 2
    for s in cache[2:]:
        s.fill_(127)
    table = (torch.arange(1 << 24, device="cuda") % pages).to(torch.int32)[None]
    q = torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda")
    out, lse = mx.cache_attention(q, cache, table, i32([(1 << 31) - 1]), scale=300 / 64, return_lse=True)
    assert mx.device_error() == 0
    assert abs(lse.item() - (-300 + math.log(2.0 ** 31))) < 2.0 ** -7 + 300 * 2.0 ** -20
    assert abs(out.float() - 2).max().item() <= 2 * (2.0 ** -6 + 2.0 ** -7)


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("sign", [-1, 1])
def test_scores_as_large_as_they_may_be(rows, sign):
    """Scores of up to 2^24 / log2 e in steps of 2^7 and more: a row takes the values of its largest one."""
    D, page, n = 64, 16, 300
    codes = 0x38 + np.random.default_rng(1).permutation(n) % 64     # 1 to 240
    k, v = np.zeros((19, 1, page, D), np.uint8), np.zeros((19, 1, page, D), np.uint8)
    for j in range(n):
        k[j // page, 0, j % page] = codes[j] | (0x80 if sign < 0 else 0)
        v[j // page, 0, j % page] = (0x30 + j % 16) | (j % 2) << 7
    bytes_ = np.full((19, 1), 127, np.uint8)
    cache = mx.KVCache(*(torch.from_numpy(x).cuda() for x in (k, v, bytes_, bytes_)))
    q = torch.ones((rows, 1, D), dtype=torch.bfloat16, device="cuda")
    scale = 2.0 ** 23 / (64 * 240)
    out, lse = mx.cache_attention(q, cache, i32(np.arange(19)[None]), i32([n]), i32([0, rows]), scale=scale, return_lse=True)
    score = sign * scale * 64 * (1 + codes % 8 / 8) * 2.0 ** (codes // 8 - 7)
    values = (1 + np.arange(n) % 8 / 8) * 2.0 ** (np.arange(n) % 16 // 8 - 1) * np.where(np.arange(n) % 2, -1, 1)
    for r in range(rows):
        seen = np.arange(n) <= n - rows + r
        best = seen & (score == score[seen].max())
        assert abs(lse[r, 0].item() / (score[best][0] + math.log(best.sum())) - 1) < 2.0 ** -21
        # Weights of keys with one score are equal: f16's and BF16's roundings are left.
        assert (out[r, 0].float() - values[best].mean()).abs().max().item() <= 2.0 ** -8 * abs(values[best].mean()) + 2.0 ** -10 * np.abs(values[best]).mean()
