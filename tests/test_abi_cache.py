"""Refusals of the rotation, cache and attention entry points: bad arguments are reported on the host before any CUDA call (so
these run without a GPU), and the binding refuses tensors of another type, device, shape or layout."""
import ctypes

import pytest
import torch

from mxfp8_block_scaled_07_b200 import build as mxbuild

A = 0x10000                        # never dereferenced: every call below fails validation first
F, ODD, BYTE = ctypes.c_void_p(A), ctypes.c_void_p(A + 8), ctypes.c_void_p(A + 1)
BIG = 1 << 31
ARG, SHAPE, ALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def mx():
    mxbuild.build()
    from mxfp8_block_scaled_07_b200 import mx

    mx.lib()
    return mx


def test_rope_table(mx):
    f = (ctypes.c_double * 128)()
    t = mx.lib().mx_rope_table
    assert t(f, 0, 1.0, 0, 4, F, None) == ARG and t(f, 4, 1.0, 0, -1, F, None) == ARG
    assert t(None, 4, 1.0, 0, 4, F, None) == ARG and t(f, 4, 1.0, 0, 4, None, None) == ARG
    assert t(f, 129, 1.0, 0, 4, F, None) == SHAPE and t(f, 4, 1.0, 0, BIG, F, None) == SHAPE
    assert t(f, 4, 1.0, 0, 4, BYTE, None) == ALIGN
    assert t(f, 4, 1.0, 0, 0, None, None) == 0


@pytest.mark.parametrize("name", ["mx_rope", "mx_rope_bwd"])
def test_rope(mx, name):
    def r(x=F, dt=1, T=4, H=2, D=64, lt=128, lh=64, tab=F, n=16, rot=32, pos=None, p64=0, y=F, yt=128, yh=64):
        return getattr(mx.lib(), name)(x, dt, T, H, D, lt, lh, tab, n, rot, pos, p64, 0, y, yt, yh, None)

    assert r(x=None) == ARG and r(y=None) == ARG and r(tab=None) == ARG and r(dt=3) == ARG and r(dt=-1) == ARG
    assert r(T=-1) == ARG and r(H=-1) == ARG and r(D=0) == ARG and r(rot=0) == ARG and r(n=-1) == ARG
    assert r(rot=33) == SHAPE and r(rot=66) == SHAPE and r(D=1025) == SHAPE and r(D=512, lh=512, yh=512, rot=258) == SHAPE
    assert r(T=17) == SHAPE and r(T=BIG, pos=F) == SHAPE and r(lh=63) == SHAPE and r(yh=-63) == SHAPE
    assert r(x=BYTE) == ALIGN and r(y=BYTE) == ALIGN and r(tab=BYTE) == ALIGN and r(dt=0, x=ctypes.c_void_p(A + 2)) == ALIGN
    assert r(pos=ctypes.c_void_p(A + 4), p64=1) == ALIGN and r(pos=BYTE) == ALIGN
    assert r(T=0, x=None, y=None, tab=None) == 0 and r(H=0, x=None, y=None) == 0


def batch(mx, **kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, k_stride=8192, v_stride=8192, ks_stride=2, vs_stride=2, pages=9, heads=2, page_size=64,
             head_dim=64, page_table=A, ld_table=4, width=4, lengths=A, row_offsets=A, sequences=3, rows=12)
    d.update(kw)
    return mx.CacheBatch(**d)


BAD_BATCHES = [(dict(pages=-1), ARG), (dict(heads=0), ARG), (dict(page_size=0), ARG), (dict(head_dim=0), ARG), (dict(width=-1), ARG),
               (dict(sequences=-1), ARG), (dict(rows=-1), ARG), (dict(lengths=None), ARG), (dict(page_table=None), ARG), (dict(k=None), ARG),
               (dict(v_scale=None), ARG), (dict(head_dim=96), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=256), SHAPE),
               (dict(heads=1025), SHAPE), (dict(rows=BIG), SHAPE), (dict(sequences=1 << 24), SHAPE), (dict(row_offsets=None), SHAPE),
               (dict(k_stride=8176), SHAPE), (dict(vs_stride=1), SHAPE), (dict(ld_table=3), SHAPE), (dict(k=A + 8), ALIGN),
               (dict(v_stride=8200), ALIGN), (dict(lengths=A + 2), ALIGN), (dict(row_offsets=A + 1), ALIGN), (dict(page_table=A + 2), ALIGN)]


def append(mx, c, k=F, kt=128, kh=64, v=F, tab=F, n=16, rot=32, q=F, Hq=4, qt=256, qh=64, o=F, ot=256, oh=64):
    return mx.lib().mx_cache_append(ctypes.byref(c) if c else None, k, kt, kh, v, 128, 64, tab, n, rot, 0, q, Hq, qt, qh, o, ot, oh, None)


def attention(mx, c, q=F, Hq=4, qt=256, qh=64, scale=0.1, o=F, ot=256, oh=64, lse=F, ws=F):
    return mx.lib().mx_cache_attention(ctypes.byref(c) if c else None, q, Hq, qt, qh, scale, 0, o, ot, oh, lse, ws, None)


@pytest.mark.parametrize("call", [append, attention])
def test_batches(mx, call):
    assert call(mx, None) == ARG
    for kw, status in BAD_BATCHES:
        assert call(mx, batch(mx, **kw)) == status, kw
    for kw in (dict(rows=0), dict(sequences=0), dict(rows=0, lengths=None, page_table=None, k=None, v=None)):
        assert call(mx, batch(mx, **kw)) == 0


def test_append(mx):
    c = batch(mx)
    assert append(mx, c, k=None) == ARG and append(mx, c, v=None) == ARG and append(mx, c, o=None) == ARG and append(mx, c, Hq=0) == ARG
    assert append(mx, c, rot=0) == ARG and append(mx, c, n=-1) == ARG
    assert append(mx, c, rot=24) == SHAPE and append(mx, c, rot=80) == SHAPE and append(mx, c, Hq=4097) == SHAPE
    assert append(mx, c, k=ODD) == ALIGN and append(mx, c, kt=132) == ALIGN and append(mx, c, kh=68) == ALIGN
    assert append(mx, c, tab=ODD) == ALIGN and append(mx, c, q=ODD) == ALIGN and append(mx, c, ot=252) == ALIGN


def test_attention(mx):
    c = batch(mx)
    assert attention(mx, c, q=None) == ARG and attention(mx, c, o=None) == ARG and attention(mx, c, ws=None) == ARG
    assert attention(mx, c, Hq=0) == ARG
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attention(mx, c, scale=scale) == ARG
    assert attention(mx, c, Hq=5) == SHAPE and attention(mx, c, Hq=4098) == SHAPE
    assert attention(mx, batch(mx, rows=BIG - 1)) == SHAPE
    assert attention(mx, c, q=ODD) == ALIGN and attention(mx, c, qh=60) == ALIGN and attention(mx, c, o=ODD) == ALIGN
    assert attention(mx, c, lse=BYTE) == ALIGN and attention(mx, c, ws=ODD) == ALIGN
    ws = mx.lib().mx_cache_attention_workspace_bytes
    assert ws(96, 4, 4) == -1 and ws(64, -1, 4) == -1 and ws(64, 4, 0) == -1 and ws(128, 0, 1) > 0


def test_binding_refuses(mx):
    """CPU tensors, wrong types, shapes and tuples, before anything is allocated or launched."""
    x, tab = torch.zeros(4, 2, 64), torch.zeros(8, 32)
    cache = mx.cache_create(2, 2, 64, 16, device="cpu")
    i = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: mx.rope(x, tab), lambda: mx.rope_backward(x, tab), lambda: mx.rope(None, tab), lambda: mx.rope(x[0], tab),
                 lambda: mx.cache_append(x, x, cache, i, i[:, 0]), lambda: mx.cache_attention(x, cache, i, i[:, 0]),
                 lambda: mx.cache_attention(x, None, i, i[:, 0]), lambda: mx.rope_table(4, 3), lambda: mx.rope_table(4, 0),
                 lambda: mx.rope_frequencies(8, 1e4, ("cubic", 2)), lambda: mx.rope_frequencies(8, 1e4, ("linear", 0)),
                 lambda: mx.rope_table(4, 8, out=torch.zeros(4, 8)), lambda: mx.cache_create(2, 2, 96), lambda: mx.cache_create(2, 2, 64, 48)):
        with pytest.raises(mx.MxError):
            call()


def test_frequencies(mx):
    f, m = mx.rope_frequencies(64, 1e4)
    assert m == 1.0 and f[0] == 1.0 and abs(f[16] - 1e-2) < 1e-15
    assert mx.rope_frequencies(64, 1e4, ("linear", 4))[0][5] == f[5] / 4
    ntk = mx.rope_frequencies(64, 1e4, ("ntk", 4))[0]
    assert ntk[0] == 1.0 and abs(ntk[31] * 4 / f[31] - 1) < 1e-12
    y, m = mx.rope_frequencies(64, 1e4, ("yarn", 4, 4096))
    assert y[0] == f[0] and abs(y[31] - f[31] / 4) < 1e-18 and abs(m - 1.1386294361119891) < 1e-15
    assert all(a / 4 <= b <= a for a, b in zip(f, y))
    assert mx.rope_frequencies(64, 1e4, ("yarn", 4, 4096, 32, 1)) == (y, m)
