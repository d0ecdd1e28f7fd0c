"""Refusals of the MXFP4 and expert-routing entry points: bad arguments are reported on the host before any CUDA
call (so these run without a GPU), and the binding refuses tensors of another type, device, shape or layout."""
import ctypes

import pytest
import torch

from mxfp8_block_scaled_07_b200 import build as mxbuild

F = ctypes.c_void_p(0x10000)       # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10008)     # not 16-byte aligned
BYTE = ctypes.c_void_p(0x10001)
BIG = 1 << 31
ARG, SHAPE, ALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    mxbuild.build()
    from mxfp8_block_scaled_07_b200 import mx

    return mx.lib()


def test_quantize_fp4(L):
    q = L.mx_quantize_fp4
    assert q(F, 64, 64, 64, 0, F, F, F, F, None) == ARG            # no direction
    assert q(F, 64, 64, 64, 8, F, F, F, F, None) == ARG            # unknown flag
    assert q(None, 64, 64, 64, 1, F, F, None, None, None) == ARG
    assert q(F, 64, 64, 64, 1, F, None, None, None, None) == ARG
    assert q(F, -1, 64, 64, 1, F, F, None, None, None) == ARG
    assert q(F, 64, 48, 64, 1, F, F, None, None, None) == SHAPE    # K % 32
    assert q(F, 48, 64, 64, 2, None, None, F, F, None) == SHAPE    # M % 32 columnwise
    assert q(F, 64, 64, 32, 1, F, F, None, None, None) == SHAPE    # ld_x < K
    assert q(ODD, 64, 64, 64, 1, F, F, None, None, None) == ALIGN
    assert q(F, 64, 64, 68, 1, F, F, None, None, None) == ALIGN
    assert q(None, 0, 64, 64, 1, None, None, None, None, None) == 0
    d = L.mx_dequantize_fp4
    assert d(F, F, -1, 64, 1, F, 64, None) == ARG
    assert d(F, None, 64, 64, 1, F, 64, None) == ARG
    assert d(F, F, 64, 40, 1, F, 64, None) == SHAPE
    assert d(F, F, 64, 64, 1, F, 32, None) == SHAPE
    assert d(F, F, 64, 64, 1, F, 68, None) == ALIGN
    assert d(F, ODD, 64, 64, 1, F, 64, None) == ALIGN              # the layout is 16-byte aligned
    assert d(None, None, 0, 64, 1, None, 64, None) == 0


def test_gemm_fp4(L):
    g = L.mx_gemm_fp4
    assert g(None, F, F, F, 8, 8, 32, F, 8, 0, None) == ARG
    assert g(F, F, F, F, 8, 8, 0, F, 8, 0, None) == ARG
    assert g(F, F, F, F, 8, 8, 32, F, 8, 7, None) == ARG
    assert g(F, F, F, F, 8, 8, 48, F, 8, 0, None) == SHAPE
    assert g(F, F, F, F, 8, 16, 32, F, 8, 0, None) == SHAPE
    assert g(F, F, F, F, 8, 8, 32, ctypes.c_void_p(0x10002), 8, 0, None) == ALIGN
    assert g(F, F, ODD, F, 8, 8, 32, F, 8, 0, None) == ALIGN
    assert g(None, None, None, None, 0, 8, 32, None, 8, 0, None) == 0
    gg = L.mx_grouped_gemm_fp4
    assert gg(F, F, F, F, None, 4, 64, 8, 32, F, 8, 0, None) == ARG
    assert gg(F, F, F, F, F, 0, 64, 8, 32, F, 8, 0, None) == ARG
    assert gg(F, F, F, F, F, 1025, 64, 8, 32, F, 8, 0, None) == SHAPE
    assert gg(F, F, F, F, BYTE, 4, 64, 8, 32, F, 8, 0, None) == ALIGN
    assert gg(F, F, F, F, F, 1024, 64, 1 << 21, 32, F, 1 << 21, 0, None) == SHAPE     # G * N


def test_route(L):
    def r(x=F, dt=0, T=4, E=8, ld=8, bias=None, score=0, groups=1, tg=1, gs=0, k=2, ids=F, w=F):
        return L.mx_route(x, dt, T, E, ld, bias, score, groups, tg, gs, k, 1, 1.0, ids, w, None)

    assert r(x=None) == ARG and r(ids=None) == ARG and r(w=None) == ARG
    assert r(T=-1) == ARG and r(E=0) == ARG and r(k=0) == ARG and r(dt=2) == ARG
    assert r(score=2) == ARG and r(gs=2) == ARG and r(groups=0) == ARG and r(tg=0) == ARG
    assert r(E=1025, ld=1025) == SHAPE and r(k=17, E=32, ld=32) == SHAPE and r(k=9) == SHAPE and r(ld=7) == SHAPE
    assert r(groups=3) == SHAPE and r(groups=2, tg=3) == SHAPE and r(E=64, ld=64, groups=64) == SHAPE
    assert r(T=BIG) == SHAPE and r(T=BIG // 2) == SHAPE
    assert r(x=ctypes.c_void_p(0x10002)) == ALIGN and r(dt=1, x=BYTE) == ALIGN
    assert r(ids=BYTE) == ALIGN and r(bias=BYTE) == ALIGN
    assert r(T=0, x=None, ids=None, w=None) == 0

    def b(dw=F, x=F, dt=0, T=4, E=8, ld=8, ids=F, score=0, k=2, out=F, ld_d=8):
        return L.mx_route_bwd(dw, x, dt, T, E, ld, ids, score, k, 1, 1.0, out, ld_d, None)

    assert b(dw=None) == ARG and b(out=None) == ARG and b(score=5) == ARG
    assert b(ld_d=7) == SHAPE and b(k=9) == SHAPE
    assert b(out=BYTE) == ALIGN
    assert b(T=0, dw=None, x=None, ids=None, out=None) == 0


def test_plan_dispatch_combine(L):
    assert L.mx_route_plan_workspace_bytes(-1, 8) == -1 and L.mx_route_plan_workspace_bytes(8, 1025) == -1
    assert L.mx_route_plan_workspace_bytes(BIG, 8) == -1 and L.mx_route_plan_workspace_bytes(100, 8) == 0
    assert L.mx_route_plan_workspace_bytes(163840, 128) > 0
    p = L.mx_route_plan
    assert p(None, 8, 4, F, F, F, None, None) == ARG and p(F, 8, 0, F, F, F, None, None) == ARG
    assert p(F, -1, 4, F, F, F, None, None) == ARG and p(F, 8, 4, F, F, None, None, None) == ARG
    assert p(F, 163840, 128, F, F, F, None, None) == ARG                    # workspace needed
    assert p(F, 8, 1025, F, F, F, None, None) == SHAPE and p(F, BIG, 4, F, F, F, F, None) == SHAPE
    assert p(BYTE, 8, 4, F, F, F, None, None) == ALIGN

    assert L.mx_grouped_scale_bytes(-1, 4, 4) == -1 and L.mx_grouped_scale_bytes(4, 0, 4) == -1
    assert L.mx_grouped_scale_bytes(0, 4, 4) == 0 and L.mx_grouped_scale_bytes(1, 8, 1) == 512
    assert L.mx_grouped_scale_bytes(3, 8, 5) == 3 * 128 * 8 and L.mx_grouped_scale_bytes(256, 1, 4) == 1024

    def d(x=F, T=4, K=64, ld=64, sr=F, k=2, off=F, E=4, fmt=0, q=F, s=F):
        return L.mx_dispatch_quantize(x, T, K, ld, sr, k, off, E, fmt, q, s, None)

    assert d(x=None) == ARG and d(sr=None) == ARG and d(off=None) == ARG and d(q=None) == ARG and d(s=None) == ARG
    assert d(fmt=2) == ARG and d(k=0) == ARG and d(E=0) == ARG and d(T=-1) == ARG
    assert d(K=48) == SHAPE and d(ld=32) == SHAPE and d(E=1025) == SHAPE and d(T=BIG // 2, k=2) == SHAPE
    assert d(x=ODD) == ALIGN and d(ld=68) == ALIGN and d(q=ODD) == ALIGN and d(s=ODD) == ALIGN and d(sr=BYTE) == ALIGN
    assert d(T=0, x=None) == 0

    def c(x=F, dt=0, rows=8, ld=16, sr=F, w=F, T=4, k=2, N=16, y=F, yt=0, ldy=16):
        return L.mx_combine(x, dt, rows, ld, sr, w, T, k, N, y, yt, ldy, None)

    assert c(x=None) == ARG and c(sr=None) == ARG and c(y=None) == ARG and c(dt=3) == ARG and c(k=0) == ARG
    assert c(ld=15) == SHAPE and c(ldy=15) == SHAPE and c(T=BIG // 2) == SHAPE and c(rows=BIG) == SHAPE
    assert c(x=ctypes.c_void_p(0x10002)) == ALIGN and c(w=BYTE) == ALIGN
    assert c(T=0, x=None) == 0

    def b(dy=F, x=F, rows=8, ld=16, sr=F, T=4, k=2, N=16, dc=F, lddc=16, dw=F, lddy=16):
        return L.mx_combine_bwd(dy, 0, lddy, x, 0, rows, ld, sr, F, T, k, N, dc, lddc, dw, None)

    assert b(dy=None) == ARG and b(x=None) == ARG and b(dc=None, dw=None) == ARG and b(sr=None) == ARG
    assert b(lddy=15) == SHAPE and b(lddc=15) == SHAPE and b(ld=15) == SHAPE
    assert b(dw=BYTE) == ALIGN


def test_binding_refuses_host_tensors_and_wrong_types(L):
    from mxfp8_block_scaled_07_b200 import mx

    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    s = torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: mx.quantize_fp4(x), lambda: mx.dequantize_fp4(u8, s), lambda: mx.gemm_fp4(u8, s, u8, s),
                 lambda: mx.grouped_gemm_fp4(u8, s, u8[None], s, ids), lambda: mx.route(x, 2),
                 lambda: mx.route(x, 2, score="relu"), lambda: mx.route_backward(x, x, ids), lambda: mx.route_plan(ids, 4),
                 lambda: mx.dispatch_quantize(x, ids, ids), lambda: mx.combine(x, ids),
                 lambda: mx.combine_backward(x, x, ids)):
        with pytest.raises(mx.MxError) as e:
            call()
        assert e.value.status == ARG
