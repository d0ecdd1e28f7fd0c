"""Calls of the rotation, cache and attention functions that are unusual but allowed, or that only look so and are refused."""
import ctypes

import numpy as np
import pytest
import torch

import plain_cache as plain
from helpers import to_np
from mxfp8_block_scaled_07_b200 import mx
from test_gpu_cache_append import i32, normal
from test_gpu_cache_attention import cache_of, verify

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


def views(buf):
    """(x, out, may be) over a buffer [20, 12, 64]: [5, 4, 64] each."""
    flat = buf.view(-1)
    packed = flat[:5 * 4 * 64].view(5, 4, 64)
    return [(buf[:5, :4], buf[:5, :4], True), (buf[:5, :4], buf[:5, 4:8], True), (buf[:5, 8:], buf[:5, :4], True), (buf[:5, :4], buf[5:10, :4], True),
            (buf[0:10:2, :4], buf[1:11:2, :4], True), (buf[0:10:2, :4], buf[0:10:2, 4:8], True),
            (buf[:5, 0:8:2], buf[:5, 1:9:2], True), (packed, flat[5 * 4 * 64:2 * 5 * 4 * 64].view(4, 5, 64).transpose(0, 1), True), (packed, buf[2:7, 4:8], True),
            (buf[:5, :4], buf[1:6, :4], False), (buf[:5, :4], buf[:5, 1:5], False), (buf[:5, :4], buf[:5, 3:7], False), (packed, flat[8:8 + 1280].view(5, 4, 64), False),
            (packed, flat[64:64 + 1280].view(5, 4, 64), False), (packed, flat[:1280].view(4, 5, 64).transpose(0, 1), False), (packed, buf[1:6, 4:8], False),
            (buf[:5, :4], buf[10:11, :4].expand(5, 4, 64), False), (buf[:5, :4], flat[8000:].as_strided((5, 4, 64), (192, 64, 1), 8000), False),
            (buf[:5, :4], flat.as_strided((5, 4, 64), (64, 192, 1), 8000), False)]


@pytest.mark.parametrize("i", range(len(views(torch.zeros(20, 12, 64)))))
def test_outputs_on_their_inputs_memory(i):
    """Outputs that are their input or lie beside it in one buffer are right; those that overlap it, or themselves, are refused and nothing is written."""
    base = normal((20, 12, 64), 1).cuda()
    cache, D, page = mx.cache_create(5, 4, 64, 16), 64, 16
    table = mx.rope_table(64, D)
    pages, lengths = i32(np.arange(5)[:, None]), i32([1, 16, 3, 9, 0])
    mx.cache_append(base[:5, :4], base[:5, 4:8], cache, pages, lengths)

    def append(x, out):
        k = base[:5, :4]
        return mx.cache_append(k, k, mx.KVCache(*(t.clone() for t in cache)), pages, lengths, q=x, table=table, out=out)

    calls = [lambda x, out: mx.rope(x, table, out=out), lambda x, out: mx.rope_backward(x, table, interleaved=True, out=out), append,
             lambda x, out: mx.cache_attention(x, cache, pages, lengths, out=out),
             lambda x, out: mx.cache_attention(x, cache, pages, lengths, i32([0, 1, 2, 5, 5, 5]), out=out)]
    for call in calls:
        buf = base.clone()
        x, out, may = views(buf)[i]
        if not may:
            with pytest.raises(mx.MxError):
                call(x, out)
            assert torch.equal(buf, base)
            continue
        want = call(x, None)
        assert torch.equal(buf, base) and call(x, out) is out and torch.equal(out, want)


def test_queries_written_over_keys_or_values_are_refused():
    buf = normal((5, 12, 64), 1).cuda()
    cache = mx.cache_create(5, 4, 64, 16)
    where = (cache, i32(np.arange(5)[:, None]), i32([1] * 5))
    for q, k, v, out in ((buf[:, :4], buf[:, 4:8], buf[:, 8:], buf[:, 4:8]), (buf[:, :4], buf[:, 4:8], buf[:, 8:], buf[:, 7:11]),
                         (buf[:, :4], buf[:, 4:8], buf[:, 8:], buf[:, 8:])):
        with pytest.raises(mx.MxError):
            mx.cache_append(k, v, *where, q=q, out=out)
    assert not cache.k.any() and not cache.v_scale.any()


@pytest.mark.parametrize("rows", [1, 30, 400])
def test_attention_over_its_queries(rows):
    """out may be q, with units of every kind: few rows and many, whole and cut."""
    lengths = np.array([rows, rows + 70, 9000])
    cache, dev, table = cache_of(lengths, 2, 128, 64, 3)
    q = normal((3 * rows, 10, 128), 1).cuda()
    where = (dev, i32(table), i32(lengths), i32(np.arange(4) * rows))
    want = mx.cache_attention(q[:, 1:9], *where)
    x = q[:, 1:9]
    assert mx.cache_attention(x, *where, out=x) is x and torch.equal(x, want)


def test_rows_named_twice_set_their_bit():
    """30 sequences that all name the same 100 rows make 60 items of 256 query rows, where 400 query rows make 10 at most: bit 2, and nothing computed."""
    cache, dev, table = cache_of([200] * 60, 1, 64, 16, 7)
    q = normal((100, 4, 64), 1).cuda()
    out = torch.full((100, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.device_error()
    mx.cache_attention(q, dev, i32(table), i32([200] * 60), i32([0, 100] * 30 + [0]), out=out)
    assert mx.device_error() == 2
    assert (out == 5).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,rows", [([1000], None), ([5, 900, 0, 17], None), ([40] * 200, None), ([700, 300], [13, 1]), ([700, 300], [300, 40]), ([64], [64]),
                                          ([9000], [257]), ([100] * 9, [100] * 9), ([20000, 300], [600, 300])])
@pytest.mark.parametrize("Hq", [2, 12])
def test_the_workspace_is_as_large_as_it_says(D, lengths, rows, Hq):
    """A workspace of exactly the bytes for the batch, between bytes that stay as they are; the same result as with the larger one of any batch."""
    Hkv, page = 2, 32
    lengths, offsets = np.array(lengths), np.concatenate([[0], np.cumsum(rows or [1] * len(lengths))])
    cache, dev, table = cache_of(lengths, Hkv, D, page, 3)
    q = normal((int(offsets[-1]), Hq, D), 1).cuda()
    t, ln, off = i32(table), i32(lengths), i32(offsets)
    c = mx.CacheBatch(dev.k.data_ptr(), dev.v.data_ptr(), dev.k_scale.data_ptr(), dev.v_scale.data_ptr(), dev.k.stride(0), dev.v.stride(0),
                      dev.k_scale.stride(0), dev.v_scale.stride(0), dev.k.shape[0], Hkv, page, D, t.data_ptr(), t.stride(0), t.shape[1], ln.data_ptr(),
                      off.data_ptr() if rows else None, len(lengths), q.shape[0])
    L, got = mx.lib(), []
    for size in (L.mx_cache_attention_batch_bytes(ctypes.byref(c), Hq), L.mx_cache_attention_workspace_bytes(D, q.shape[0], Hq)):
        space = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        assert L.mx_cache_attention(ctypes.byref(c), q.data_ptr(), Hq, Hq * D, D, D ** -0.5, 0, out.data_ptr(), Hq * D, D, None, space.data_ptr() + 4096,
                                    torch.cuda.current_stream().cuda_stream) == 0
        assert (space[:4096] == 0xA5).all() and (space[4096 + size:] == 0xA5).all()
        got.append(out)
    assert mx.device_error() == 0 and torch.equal(got[0], got[1])
    assert torch.equal(got[0], mx.cache_attention(q, dev, t, ln, off if rows else None))
    verify(got[0], None, q, cache, table, lengths, offsets, D ** -0.5, 0, D)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("H,D,rot,gap", [(1, 64, 32, 0), (9, 128, 64, 0), (3, 80, 16, 8), (5, 30, 14, 0), (2, 129, 128, 1), (40, 96, 96, 0), (1, 1024, 2, 0)])
def test_padding_tokens_in_place(H, D, rot, gap, dtype, interleaved, back):
    """A token of a negative position or one behind the table is zeros whole, rotated in place as elsewhere; gaps between heads stay."""
    T = 6
    f = mx.rope_backward if back else mx.rope
    table = torch.from_numpy(plain.table(10, plain.frequencies(rot))).cuda()
    pos = torch.tensor([3, -1, 9, 10, 0, -7], device="cuda")
    buf = normal((T, H, D + gap), 1).to(dtype).cuda()
    x = buf[:, :, :D]
    want, rest = f(x, table, pos, interleaved), buf[:, :, D:].clone()
    assert not want[1].any() and not want[3].any() and not want[5].any() and want[2, :, rot:].equal(x[2, :, rot:])
    assert f(x, table, pos, interleaved, out=x) is x
    assert torch.equal(x, want) and torch.equal(buf[:, :, D:], rest) and mx.device_error() == 4
