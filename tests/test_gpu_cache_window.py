"""Attention with a window leaves pages in front of it alone: a sampler gives them to other sequences and marks their entries."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32, normal
from test_gpu_cache_attention import cache_of, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [1, 33, 50, 1024])
@pytest.mark.parametrize("rows,D", [(1, 128), (12, 64), (100, 128), (300, 64)])
def test_released_pages(rows, D, window, page):
    """Entries of pages that no row sees are -1: no error, and the outputs are those of the whole table."""
    Hkv, G = 2, 3
    lengths = np.array([rows, rows + 70, 1500, 2000, 2049 + rows])
    cache, dev, table = cache_of(lengths, Hkv, D, page, window)
    offsets = np.arange(len(lengths) + 1) * rows
    q = normal((int(offsets[-1]), Hkv * G, D), 1).cuda()
    released = table.copy()
    for b, n in enumerate(lengths):
        released[b, :max(n - rows - window + 1, 0) // page] = -1
    for off in (i32(offsets),) + ((None,) if rows == 1 else ()):
        want, want_lse = mx.cache_attention(q, dev, i32(table), i32(lengths), off, window=window, return_lse=True)
        assert mx.device_error() == 0
        got, lse = mx.cache_attention(q, dev, i32(released), i32(lengths), off, window=window, return_lse=True)
        assert mx.device_error() == 0
        assert torch.equal(got, want) and torch.equal(lse, want_lse)
    verify(got, lse, q, cache, table, lengths, offsets, D ** -0.5, window, D)
