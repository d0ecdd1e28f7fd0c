"""Calls of the rotation, cache and attention functions that are unusual but allowed, or that only look so and are refused."""
import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("single", [True, False])
def test_a_rotation_table_without_positions(single):
    """Every position lies behind it: zeros and bit 4, as rope() has it, and not keys as they are."""
    H, D, page, n = 2, 64, 16, 3
    cache = mx.cache_create(n, H, D, page)
    k, v, q = normal((n, H, D), 1), normal((n, H, D), 2), normal((n, 4, D), 3)
    table = torch.zeros((0, D), device="cuda")
    pages, lengths, offsets = np.arange(n)[:, None], np.array([5, 1, 16]), np.arange(n + 1)
    mx.device_error()
    out = mx.cache_append(k.cuda(), v.cuda(), cache, i32(pages), i32(lengths), None if single else i32(offsets), q=q.cuda(), table=table)
    assert mx.device_error() == 4
    assert not out.any()
    for x, code, byte in ((np.zeros((n, H, D)), cache.k, cache.k_scale), (v.double().numpy(), cache.v, cache.v_scale)):
        want = plain.append((np.zeros((n, H, page, D), np.uint8), np.zeros((n, H), np.uint8)), x, pages, lengths, offsets)
        assert np.array_equal(to_np(code), want[0]) and np.array_equal(to_np(byte), want[1])
    assert not mx.rope(q.cuda(), table, i32(lengths)).any() and mx.device_error() == 4
