"""Attention at the ends of what its arguments may be: as many tokens as an int32 counts."""
import math

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
