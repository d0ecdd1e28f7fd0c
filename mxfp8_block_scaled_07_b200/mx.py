"""Thin Python binding of libmx (include/mx.h) over ctypes.

Argument marshalling only: every step runs in the CUDA kernels of ``libmx.so``. PyTorch
supplies device memory (output tensors are allocated with ``torch.empty`` on the input's
device) and the current stream. There is no fallback: if ``libmx.so`` is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmx.so")

MX_ROWWISE, MX_COLWISE, MX_SWIZZLE = 1, 2, 4
MX_OUT_F32, MX_OUT_BF16 = 0, 1
MX_SCORE = {"softmax": 0, "sigmoid": 1}
MX_GROUP = {"max": 0, "top2": 1}
MX_FORMAT = {"mxfp8": 0, "mxfp4": 1}
_STATUS = {0: "MX_OK", -1: "MX_ERR_ARG", -2: "MX_ERR_SHAPE", -3: "MX_ERR_ALIGN", -4: "MX_ERR_CUDA",
           -5: "MX_ERR_UNSUPPORTED", -6: "MX_ERR_DEVICE"}

_lib = None


class QuantTensor(ctypes.Structure):
    """mx_quant_tensor."""
    _fields_ = [("x", ctypes.c_void_p), ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("q_row", ctypes.c_void_p), ("s_row", ctypes.c_void_p), ("q_col", ctypes.c_void_p),
                ("s_col", ctypes.c_void_p)]


class GridRef(ctypes.Structure):
    """mx_grid_ref."""
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class ComparePair(ctypes.Structure):
    """mx_compare_pair."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("nbytes", ctypes.c_int64)]


class MxError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libmx.so with argument types declared (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmx.so not built ({LIB_PATH}); run python -m mxfp8_block_scaled_07_b200.build")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
    L.mx_swizzled_scale_bytes.argtypes = [I64, I64]
    L.mx_swizzled_scale_bytes.restype = I64
    L.mx_quantize.argtypes = [P, I64, I64, I64, I32, P, P, P, P, P]
    L.mx_quantize.restype = I32
    L.mx_swizzle_scales.argtypes = [P, I64, I64, P, I64, P, P]
    L.mx_swizzle_scales.restype = I32
    L.mx_gemm.argtypes = [P, P, P, P, I64, I64, I64, P, I64, I32, P]
    L.mx_gemm.restype = I32
    L.mx_quantize_block128.argtypes = [P, I64, I64, I64, I32, P, P, P]
    L.mx_quantize_block128.restype = I32
    L.mx_grouped_gemm_swiglu_quant.argtypes = [P, P, P, P, P, I64, I64, I64, I64, P, P, P]
    L.mx_grouped_gemm_swiglu_quant.restype = I32
    L.mx_grouped_gemm.argtypes = [P, P, P, P, P, I64, I64, I64, I64, P, I64, I32, P]
    L.mx_grouped_gemm.restype = I32
    L.mx_grid_equal.argtypes = [P, P, I64, P, P, P]
    L.mx_grid_equal.restype = I32
    L.mx_quantize_multi.argtypes = [P, I64, I32, P]
    L.mx_quantize_multi.restype = I32
    L.mx_grid_equal_multi.argtypes = [P, I64, P, P, P]
    L.mx_grid_equal_multi.restype = I32
    L.mx_quantize_compare_multi.argtypes = [P, P, I64, P, P, P]
    L.mx_quantize_compare_multi.restype = I32
    F32 = ctypes.c_float
    for name, args in (
            ("mx_quantize_fp4", [P, I64, I64, I64, I32, P, P, P, P, P]),
            ("mx_dequantize_fp4", [P, P, I64, I64, I32, P, I64, P]),
            ("mx_gemm_fp4", [P, P, P, P, I64, I64, I64, P, I64, I32, P]),
            ("mx_grouped_gemm_fp4", [P, P, P, P, P, I64, I64, I64, I64, P, I64, I32, P]),
            ("mx_route", [P, I32, I64, I64, I64, P, I32, I64, I64, I32, I64, I32, F32, P, P, P]),
            ("mx_route_bwd", [P, P, I32, I64, I64, I64, P, I32, I64, I32, F32, P, I64, P]),
            ("mx_route_plan", [P, I64, I64, P, P, P, P, P]),
            ("mx_dispatch_quantize", [P, I64, I64, I64, P, I64, P, I64, I32, P, P, P]),
            ("mx_combine", [P, I32, I64, I64, P, P, I64, I64, I64, P, I32, I64, P]),
            ("mx_combine_bwd", [P, I32, I64, P, I32, I64, I64, P, P, I64, I64, I64, P, I64, P, P])):
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = I32
    L.mx_route_plan_workspace_bytes.argtypes = [I64, I64]
    L.mx_route_plan_workspace_bytes.restype = I64
    L.mx_grouped_scale_bytes.argtypes = [I64, I64, I64]
    L.mx_grouped_scale_bytes.restype = I64
    L.mx_status_string.argtypes = [I32]
    L.mx_status_string.restype = ctypes.c_char_p
    L.mx_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.mx_device_error.restype = I32
    L.mx_set_wait_timeout_ns.argtypes = [U64]
    L.mx_set_wait_timeout_ns.restype = None
    L.mx_set_gemm_variant.argtypes = [I32]
    L.mx_set_gemm_variant.restype = None
    L.mx_set_quantize_variant.argtypes = [I32]
    L.mx_set_quantize_variant.restype = None
    L.mx_diag_expired_wait.argtypes = [P]
    L.mx_diag_expired_wait.restype = I32
    _lib = L
    return L


def _check(status: int, what: str):
    if status != 0:
        raise MxError(status, what)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def swizzled_scale_bytes(rows: int, kblocks: int) -> int:
    return int(lib().mx_swizzled_scale_bytes(rows, kblocks))


def grouped_swizzled_scale_bytes(group_rows, kblocks: int) -> int:
    """Bytes of the grouped layout: every group padded to 128 rows on its own (no library call per
    group: the padded row count times the padded K-block count)."""
    rows = sum((int(r) + 127) // 128 * 128 for r in group_rows)
    return swizzled_scale_bytes(rows, kblocks) if rows else 0


def quantize(x: torch.Tensor, rowwise: bool = True, colwise: bool = False, swizzle: bool = True, out=None):
    """mx_quantize on a 2-D BF16 CUDA tensor. Returns (q_row, s_row, q_col, s_col); entries of a
    direction not requested are None. ``out`` may supply the four buffers."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    flags = (MX_ROWWISE if rowwise else 0) | (MX_COLWISE if colwise else 0) | (MX_SWIZZLE if swizzle else 0)
    dev = x.device
    if out is None:
        u8 = dict(dtype=torch.uint8, device=dev)
        q_row = torch.empty((M, K), **u8) if rowwise else None
        s_row = (torch.empty(swizzled_scale_bytes(M, K // 32), **u8) if swizzle
                 else torch.empty((M, K // 32), **u8)) if rowwise else None
        q_col = torch.empty((K, M), **u8) if colwise else None
        s_col = (torch.empty(swizzled_scale_bytes(K, M // 32), **u8) if swizzle
                 else torch.empty((K, M // 32), **u8)) if colwise else None
    else:
        q_row, s_row, q_col, s_col = out
    st = lib().mx_quantize(_p(x), M, K, x.stride(0), flags, _p(q_row), _p(s_row), _p(q_col), _p(s_col),
                           ctypes.c_void_p(_stream(dev)))
    _check(st, "mx_quantize")
    return q_row, s_row, q_col, s_col


def quant_tensor_array(xs, outs):
    """ctypes array of mx_quant_tensor for tensors xs and their (q_row, s_row, q_col, s_col) outputs."""
    arr = (QuantTensor * len(xs))()
    for i, (x, (q_row, s_row, q_col, s_col)) in enumerate(zip(xs, outs)):
        assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
        arr[i] = QuantTensor(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0),
                             *(t.data_ptr() if t is not None else None for t in (q_row, s_row, q_col, s_col)))
    return arr


def quantize_multi(xs, rowwise: bool = True, colwise: bool = False, swizzle: bool = True, outs=None):
    """mx_quantize_multi over a list of 2-D BF16 CUDA tensors (same flags); returns one
    (q_row, s_row, q_col, s_col) tuple per tensor."""
    if outs is None:
        outs = []
        for x in xs:
            M, K = x.shape
            u8 = dict(dtype=torch.uint8, device=x.device)
            outs.append((
                torch.empty((M, K), **u8) if rowwise else None,
                (torch.empty(swizzled_scale_bytes(M, K // 32), **u8) if swizzle else torch.empty((M, K // 32), **u8))
                if rowwise else None,
                torch.empty((K, M), **u8) if colwise else None,
                (torch.empty(swizzled_scale_bytes(K, M // 32), **u8) if swizzle else torch.empty((K, M // 32), **u8))
                if colwise else None))
    flags = (MX_ROWWISE if rowwise else 0) | (MX_COLWISE if colwise else 0) | (MX_SWIZZLE if swizzle else 0)
    arr = quant_tensor_array(xs, outs)
    dev = xs[0].device if xs else torch.device("cuda")
    st = lib().mx_quantize_multi(ctypes.cast(arr, ctypes.c_void_p), len(xs), flags, ctypes.c_void_p(_stream(dev)))
    _check(st, "mx_quantize_multi")
    return outs


def compare_pair_array(pairs):
    arr = (ComparePair * len(pairs))()
    for i, (a, b) in enumerate(pairs):
        n = a.numel() * a.element_size()
        assert a.is_contiguous() and b.is_contiguous() and b.numel() * b.element_size() == n
        arr[i] = ComparePair(a.data_ptr(), b.data_ptr(), n)
    return arr


def quantize_compare_multi(xs, refs, outs=None, results=None):
    """mx_quantize_compare_multi: the rowwise codes and tensor-core scale layout of every BF16
    tensor in xs (written to outs, as quantize_multi(xs, True, False, True) would), compared byte for
    byte with refs[i] = (q, s_swizzled) in the same pass. Returns (outs, mismatches, first_index);
    the last two are int64 device tensors of 2 len(xs) entries: codes then scales per tensor."""
    n = len(xs)
    dev = xs[0].device if xs else torch.device("cuda")
    if outs is None:
        outs = []
        for x in xs:
            M, K = x.shape
            u8 = dict(dtype=torch.uint8, device=x.device)
            outs.append((torch.empty((M, K), **u8), torch.empty(swizzled_scale_bytes(M, K // 32), **u8), None, None))
    if results is None:
        results = torch.empty((2, max(2 * n, 1)), dtype=torch.int64, device=dev)
    arr = quant_tensor_array(xs, outs)
    ref_arr = (GridRef * max(n, 1))()
    for i, (q, s) in enumerate(refs):
        ref_arr[i] = GridRef(q.data_ptr(), s.data_ptr())
    st = lib().mx_quantize_compare_multi(ctypes.cast(arr, ctypes.c_void_p), ctypes.cast(ref_arr, ctypes.c_void_p), n,
                                         _p(results[0]), _p(results[1]), ctypes.c_void_p(_stream(dev)))
    _check(st, "mx_quantize_compare_multi")
    return outs, results[0, :2 * n], results[1, :2 * n]


def grid_equal_multi(pairs, out=None):
    """mx_grid_equal_multi over a list of (a, b) CUDA tensor pairs. Returns (mismatches, first_index):
    int64 device tensors of len(pairs) entries (no host synchronisation)."""
    n = len(pairs)
    dev = pairs[0][0].device if pairs else torch.device("cuda")
    if out is None:
        out = torch.empty((2, max(n, 1)), dtype=torch.int64, device=dev)
    arr = compare_pair_array(pairs)
    st = lib().mx_grid_equal_multi(ctypes.cast(arr, ctypes.c_void_p), n, _p(out[0]), _p(out[1]),
                                   ctypes.c_void_p(_stream(dev)))
    _check(st, "mx_grid_equal_multi")
    return out[0, :n], out[1, :n]


def swizzle_scales(s: torch.Tensor, group_rows=None, out=None):
    """mx_swizzle_scales on raw scales [rows, kblocks] (uint8, CUDA)."""
    assert s.dtype == torch.uint8 and s.dim() == 2 and s.is_contiguous()
    rows, kb = s.shape
    if group_rows is not None:
        gr = np.ascontiguousarray(np.asarray(group_rows, dtype=np.int64))       # host memory, read during the call
        gptr, ng = ctypes.c_void_p(gr.ctypes.data), int(gr.size)
    else:
        gr, gptr, ng = None, None, 0
    if out is None:
        size = grouped_swizzled_scale_bytes(gr, kb) if gr is not None else swizzled_scale_bytes(rows, kb)
        out = torch.empty(size, dtype=torch.uint8, device=s.device)
    st = lib().mx_swizzle_scales(_p(s), rows, kb, gptr, ng, _p(out), ctypes.c_void_p(_stream(s.device)))
    _check(st, "mx_swizzle_scales")
    return out


_OUT_CODES = {torch.float32: MX_OUT_F32, torch.bfloat16: MX_OUT_BF16}


def _out_code(dtype) -> int:
    return _OUT_CODES[dtype]


def gemm(qa, sa_swz, qb, sb_swz, out_dtype=torch.bfloat16, out=None):
    """mx_gemm: C[M, N] = A . B^T from K-major E4M3 operands and tensor-core-layout scales."""
    M, K = qa.shape
    N = qb.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=qa.device)
    st = lib().mx_gemm(_p(qa), _p(sa_swz), _p(qb), _p(sb_swz), M, N, K, _p(out), out.stride(0),
                       _out_code(out.dtype), ctypes.c_void_p(_stream(qa.device)))
    _check(st, "mx_gemm")
    return out


def grouped_gemm(qa, sa_swz, qb, sb_swz, row_offsets, out_dtype=torch.bfloat16, out=None):
    """mx_grouped_gemm: rows [off[g], off[g+1]) of A against qb[g]. row_offsets: int32 CUDA [G+1]."""
    total, K = qa.shape
    G, N, K2 = qb.shape
    assert K2 == K and row_offsets.dtype == torch.int32 and row_offsets.numel() == G + 1
    if out is None:
        out = torch.empty((total, N), dtype=out_dtype, device=qa.device)
    st = lib().mx_grouped_gemm(_p(qa), _p(sa_swz), _p(qb), _p(sb_swz), _p(row_offsets), G, total, N, K, _p(out),
                               out.stride(0), _out_code(out.dtype), ctypes.c_void_p(_stream(qa.device)))
    _check(st, "mx_grouped_gemm")
    return out


def grouped_gemm_swiglu_quant(qa, sa_swz, qb, sb_swz, row_offsets, group_rows, out=None):
    """mx_grouped_gemm_swiglu_quant. qb: [G, 2 n, K] with gate/up rows interleaved per 128;
    group_rows: rows per expert (host), for the size of h's grouped scale layout. Returns
    (h_q uint8 [total, n], h_s uint8 grouped tensor-core layout of [total, n / 32])."""
    total, K = qa.shape
    G, N2, K2 = qb.shape
    assert K2 == K and N2 % 2 == 0 and row_offsets.dtype == torch.int32 and row_offsets.numel() == G + 1
    n = N2 // 2
    if out is None:
        u8 = dict(dtype=torch.uint8, device=qa.device)
        out = (torch.empty((total, n), **u8),
               torch.empty(grouped_swizzled_scale_bytes([int(r) for r in group_rows], n // 32), **u8))
    hq, hs = out
    st = lib().mx_grouped_gemm_swiglu_quant(_p(qa), _p(sa_swz), _p(qb), _p(sb_swz), _p(row_offsets), G, total, n,
                                            K, _p(hq), _p(hs), ctypes.c_void_p(_stream(qa.device)))
    _check(st, "mx_grouped_gemm_swiglu_quant")
    return hq, hs


def quantize_block128(x: torch.Tensor, pow2_scales: bool, out=None):
    """mx_quantize_block128 on a 2-D BF16 CUDA tensor: FP8 blockwise codes with one FP32
    (pow2_scales=False) or power-of-two (pow2_scales=True) scale per 128 x 128 block.
    Returns (q uint8 [M, K], scales float32 [ceil(M/128), ceil(K/128)])."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        out = (torch.empty((M, K), dtype=torch.uint8, device=x.device),
               torch.empty(((M + 127) // 128, (K + 127) // 128), dtype=torch.float32, device=x.device))
    q, sc = out
    st = lib().mx_quantize_block128(_p(x), M, K, x.stride(0), 1 if pow2_scales else 0, _p(q), _p(sc),
                                    ctypes.c_void_p(_stream(x.device)))
    _check(st, "mx_quantize_block128")
    return q, sc


# ---- MXFP4 and expert routing: tensors are checked here (type, device, layout), sizes by the library ----

def _need(ok: bool, what: str):
    if not ok:
        raise MxError(-1, what)


# (Attribute checks in the order of their cost; anything that is no tensor fails them too. A host tensor is refused by
# _call(), which every function ends in, or by the device check against the first operand.)

def _matrix(t, what: str, dtypes, shape=None, dev=None) -> int:
    """Checks a 2-D CUDA tensor with unit column stride (and its shape and device); returns its address."""
    try:
        ok = (t.dtype in dtypes and t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1)
              and (t.is_cuda if dev is None else t.device == dev) and (shape is None or t.shape == shape))
    except AttributeError:
        ok = False
    if not ok:
        raise MxError(-1, what)
    return t.data_ptr()


def _packed(t, what: str, dtype, numel: int, dev) -> int:
    """Checks a contiguous tensor of `numel` elements on `dev`; returns its address."""
    try:
        ok = t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.device == dev
    except AttributeError:
        ok = False
    if not ok:
        raise MxError(-1, what)
    return t.data_ptr()


def _layout_bytes(rows: int, kblocks: int) -> int:
    """mx_swizzled_scale_bytes without the library call (for sizes known to be >= 0)."""
    return (rows + 127) // 128 * 128 * ((kblocks + 3) // 4 * 4)


def _ld(t) -> int:
    """Row stride in elements. Of a single row no stride is ever used: its own width stands for it."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


# The current stream's handle without a Stream object around it: half a call's Python time where a call takes 10 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(name: str, dev, *args):
    """One library call on `dev`'s current stream, with `dev` as the current device."""
    fn = getattr(_lib or lib(), name)
    i = dev.index
    if dev.type != "cuda":
        raise MxError(-1, f"{name}: CUDA tensors")
    if i == torch.cuda.current_device():
        st = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = fn(*args, _raw_stream(i))
    if st != 0:
        raise MxError(st, name)


_FLOATS = (torch.float32, torch.bfloat16)
_U8, _BF16, _I32, _F32 = (torch.uint8,), (torch.bfloat16,), (torch.int32,), (torch.float32,)


def quantize_fp4(x: torch.Tensor, rowwise: bool = True, colwise: bool = False, swizzle: bool = True, out=None):
    """mx_quantize_fp4 on a 2-D BF16 CUDA tensor. Returns (q_row [M, K/2], s_row, q_col [K, M/2], s_col), uint8;
    two E2M1 codes per byte, the even element in the low four bits; scales as quantize() gives them. Entries of a
    direction not requested are None. ``out`` may supply the four buffers."""
    px = _matrix(x, "quantize_fp4: x must be a 2-D BF16 CUDA tensor with unit column stride", _BF16)
    M, K = x.shape
    dev = x.device
    flags = (MX_ROWWISE if rowwise else 0) | (MX_COLWISE if colwise else 0) | (MX_SWIZZLE if swizzle else 0)

    def scale_bytes(rows, n):
        return _layout_bytes(rows, n // 32) if swizzle else rows * (n // 32)

    if out is None:
        _need(K % 32 == 0 and (not colwise or M % 32 == 0), "quantize_fp4: blocks of 32 along the quantized axis")
        new = x.new_empty
        q_row = new((M, K // 2), dtype=torch.uint8) if rowwise else None
        s_row = new(scale_bytes(M, K) if swizzle else (M, K // 32), dtype=torch.uint8) if rowwise else None
        q_col = new((K, M // 2), dtype=torch.uint8) if colwise else None
        s_col = new(scale_bytes(K, M) if swizzle else (K, M // 32), dtype=torch.uint8) if colwise else None
        p = [None if t is None else t.data_ptr() for t in (q_row, s_row, q_col, s_col)]
    else:
        q_row, s_row, q_col, s_col = out
        p = [None] * 4
        if rowwise:
            p[0] = _packed(q_row, "quantize_fp4: q_row", torch.uint8, M * K // 2, dev)
            p[1] = _packed(s_row, "quantize_fp4: s_row", torch.uint8, scale_bytes(M, K), dev)
        if colwise:
            p[2] = _packed(q_col, "quantize_fp4: q_col", torch.uint8, M * K // 2, dev)
            p[3] = _packed(s_col, "quantize_fp4: s_col", torch.uint8, scale_bytes(K, M), dev)
    _call("mx_quantize_fp4", dev, px, M, K, _ld(x), flags, *p)
    return q_row, s_row, q_col, s_col


def dequantize_fp4(q: torch.Tensor, s: torch.Tensor, swizzled: bool = True, out=None):
    """mx_dequantize_fp4: the BF16 values [M, K] of packed codes q [M, K/2] and their scales (the tensor-core
    layout, or raw [M, K/32] with swizzled=False)."""
    dev = q.device
    _need(isinstance(q, torch.Tensor) and q.dim() == 2, "dequantize_fp4: q must be a 2-D uint8 CUDA tensor")
    M, K = q.shape[0], 2 * q.shape[1]
    pq = _packed(q, "dequantize_fp4: q must be a contiguous uint8 CUDA tensor", torch.uint8, M * K // 2, dev)
    ps = _packed(s, "dequantize_fp4: s", torch.uint8, _layout_bytes(M, K // 32) if swizzled else M * (K // 32), dev)
    if out is None:
        out = q.new_empty((M, K), dtype=torch.bfloat16)
    _call("mx_dequantize_fp4", dev, pq, ps, M, K, int(swizzled), _matrix(out, "dequantize_fp4: out", _BF16, (M, K), dev),
          _ld(out))
    return out


def gemm_fp4(qa, sa_swz, qb, sb_swz, out_dtype=torch.bfloat16, out=None):
    """mx_gemm_fp4: C[M, N] = A . B^T from packed K-major E2M1 operands (qa [M, K/2], qb [N, K/2]) and
    tensor-core-layout scales."""
    dev = qa.device
    _need(qa.dim() == 2 and qb.dim() == 2 and qa.shape[1] == qb.shape[1], "gemm_fp4: qa [M, K/2] and qb [N, K/2]")
    (M, K), N = qa.shape, qb.shape[0]
    K *= 2
    pa = _packed(qa, "gemm_fp4: qa", torch.uint8, M * K // 2, dev)
    pb = _packed(qb, "gemm_fp4: qb", torch.uint8, N * K // 2, dev)
    psa = _packed(sa_swz, "gemm_fp4: sa_swz", torch.uint8, _layout_bytes(M, K // 32), dev)
    psb = _packed(sb_swz, "gemm_fp4: sb_swz", torch.uint8, _layout_bytes(N, K // 32), dev)
    if out is None:
        out = qa.new_empty((M, N), dtype=out_dtype)
    _call("mx_gemm_fp4", dev, pa, psa, pb, psb, M, N, K, _matrix(out, "gemm_fp4: out", _FLOATS, (M, N), dev), _ld(out),
          _out_code(out.dtype))
    return out


def grouped_gemm_fp4(qa, sa_swz, qb, sb_swz, row_offsets, out_dtype=torch.bfloat16, out=None):
    """mx_grouped_gemm_fp4: rows [off[g], off[g+1]) of A (packed [rows, K/2]) against qb[g] ([G, N, K/2] packed,
    sb_swz G consecutive layouts). sa_swz: A's grouped layout, at least as many bytes as the groups' rows need
    (grouped_scale_bytes_bound() always suffices). row_offsets: int32 CUDA [G + 1]."""
    dev = qa.device
    _need(qa.dim() == 2 and qb.dim() == 3 and qb.shape[2] == qa.shape[1], "grouped_gemm_fp4: qa [rows, K/2] and qb [G, N, K/2]")
    rows, K = qa.shape[0], 2 * qa.shape[1]
    G, N = qb.shape[0], qb.shape[1]
    pa = _packed(qa, "grouped_gemm_fp4: qa must be contiguous", torch.uint8, rows * K // 2, dev)
    pb = _packed(qb, "grouped_gemm_fp4: qb", torch.uint8, G * N * K // 2, dev)
    psb = _packed(sb_swz, "grouped_gemm_fp4: sb_swz", torch.uint8, G * _layout_bytes(N, K // 32), dev)
    _need(isinstance(sa_swz, torch.Tensor) and sa_swz.numel() >= _layout_bytes(rows, K // 32), "grouped_gemm_fp4: sa_swz")
    psa = _packed(sa_swz, "grouped_gemm_fp4: sa_swz", torch.uint8, sa_swz.numel(), dev)
    poff = _packed(row_offsets, "grouped_gemm_fp4: row_offsets must be int32 [G + 1]", torch.int32, G + 1, dev)
    if out is None:
        out = qa.new_empty((rows, N), dtype=out_dtype)
    _call("mx_grouped_gemm_fp4", dev, pa, psa, pb, psb, poff, G, rows, N, K,
          _matrix(out, "grouped_gemm_fp4: out", _FLOATS, (rows, N), dev), _ld(out), _out_code(out.dtype))
    return out


def route(logits: torch.Tensor, topk: int, score: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
          group_score: str = "max", renormalize: bool = True, scale: float = 1.0, out=None):
    """mx_route: the topk experts of every token and their weights from router logits [T, E] (fp32 or BF16).

    score: "softmax" or "sigmoid"; bias: fp32 [E] added to the scores for the choice only; groups, topk_groups,
    group_score ("max" or "top2"): experts outside the best groups are left out; weights are scale * score, over the
    chosen experts' sum if renormalize. Returns (ids int32 [T, topk], weights fp32 [T, topk]); id -1 and weight 0
    where no expert is left (logits of -inf or NaN take an expert out)."""
    p = _matrix(logits, "route: logits must be a 2-D fp32 or BF16 CUDA tensor with unit column stride", _FLOATS)
    _need(score in MX_SCORE and group_score in MX_GROUP, "route: score is 'softmax' or 'sigmoid', group_score 'max' or 'top2'")
    T, E = logits.shape
    dev = logits.device
    pb = None if bias is None else _packed(bias, "route: bias must be fp32 [E]", torch.float32, E, dev)
    if out is None:
        _need(topk >= 1, "route: topk")
        ids, weights = logits.new_empty((T, topk), dtype=torch.int32), logits.new_empty((T, topk), dtype=torch.float32)
        pi, pw = ids.data_ptr(), weights.data_ptr()
    else:
        ids, weights = out
        pi = _packed(ids, "route: ids must be int32 [T, topk]", torch.int32, T * topk, dev)
        pw = _packed(weights, "route: weights must be fp32 [T, topk]", torch.float32, T * topk, dev)
    _call("mx_route", dev, p, _out_code(logits.dtype), T, E, _ld(logits), pb, MX_SCORE[score], groups, topk_groups,
          MX_GROUP[group_score], topk, int(renormalize), scale, pi, pw)
    return ids, weights


def route_backward(d_weights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0, out=None):
    """mx_route_bwd: the gradient of route()'s weights with respect to the logits, the choice (ids) held fixed."""
    p = _matrix(logits, "route_backward: logits must be a 2-D fp32 or BF16 CUDA tensor with unit column stride", _FLOATS)
    _need(score in MX_SCORE and ids.dim() == 2, "route_backward: score is 'softmax' or 'sigmoid', ids [T, topk]")
    T, E = logits.shape
    dev, topk = logits.device, ids.shape[1]
    if out is None:
        out = logits.new_empty((T, E))
    _call("mx_route_bwd", dev, _packed(d_weights, "route_backward: d_weights must be fp32 [T, topk]", torch.float32, T * topk, dev),
          p, _out_code(logits.dtype), T, E, _ld(logits), _packed(ids, "route_backward: ids must be int32 [T, topk]", torch.int32, T * topk, dev),
          MX_SCORE[score], topk, int(renormalize), scale, _matrix(out, "route_backward: out", (logits.dtype,), (T, E), dev), _ld(out))
    return out


def route_plan(ids: torch.Tensor, experts: int, out=None):
    """mx_route_plan: (row_offsets int32 [experts + 1], slot_row int32 like ids, counts int32 [experts]) of the
    experts' ids [T, topk]. row_offsets always ends at ids.numel(): slots without an expert are padding rows of the
    last group, and their slot_row is ~row."""
    _need(isinstance(ids, torch.Tensor) and ids.is_cuda, "route_plan: ids must be an int32 CUDA tensor")
    dev, n = ids.device, ids.numel()
    p = _packed(ids, "route_plan: ids must be a contiguous int32 tensor", torch.int32, n, dev)
    size = int(lib().mx_route_plan_workspace_bytes(n, experts))
    _need(size >= 0, "route_plan: 1 to 1024 experts")
    if out is None:
        off, slot_row, counts = ids.new_empty(experts + 1), torch.empty_like(ids), ids.new_empty(experts)
        po, ps, pc = off.data_ptr(), slot_row.data_ptr(), counts.data_ptr()
    else:
        off, slot_row, counts = out
        po = _packed(off, "route_plan: row_offsets must be int32 [experts + 1]", torch.int32, experts + 1, dev)
        ps = _packed(slot_row, "route_plan: slot_row must be int32 like ids", torch.int32, n, dev)
        pc = _packed(counts, "route_plan: counts must be int32 [experts]", torch.int32, experts, dev)
    ws = ids.new_empty(size, dtype=torch.uint8) if size else None
    _call("mx_route_plan", dev, p, n, experts, po, ps, pc, None if ws is None else ws.data_ptr())
    return off, slot_row, counts


def grouped_scale_bytes_bound(rows: int, groups: int, kblocks: int) -> int:
    """mx_grouped_scale_bytes: bytes that hold the grouped scale layout of any split of `rows` into `groups` (-1 for bad
    sizes)."""
    if rows < 0 or groups < 1 or kblocks < 0:
        return -1
    return (rows + 127 * min(groups, rows)) // 128 * 128 * ((kblocks + 3) // 4 * 4)


def dispatch_quantize(x: torch.Tensor, slot_row: torch.Tensor, row_offsets: torch.Tensor, fmt: str = "mxfp8", out=None):
    """mx_dispatch_quantize: tokens x [T, K] (BF16) quantized into the experts' rows that route_plan() laid out.
    Returns (q, s): uint8 codes [T * topk, K] ("mxfp8") or [T * topk, K/2] ("mxfp4") and the grouped scale layout
    (grouped_scale_bytes_bound() bytes, zeros where no row lies): the A operand of the grouped products."""
    p = _matrix(x, "dispatch_quantize: x must be a 2-D BF16 CUDA tensor with unit column stride", _BF16)
    _need(fmt in MX_FORMAT and slot_row.dim() == 2 and slot_row.shape[0] == x.shape[0] and row_offsets.numel() >= 2,
          "dispatch_quantize: fmt is 'mxfp8' or 'mxfp4', slot_row [T, topk], row_offsets [E + 1]")
    T, K = x.shape
    dev, topk, E = x.device, slot_row.shape[1], row_offsets.numel() - 1
    width = K if fmt == "mxfp8" else K // 2
    size = max(grouped_scale_bytes_bound(T * topk, E, K // 32), 0)
    if out is None:
        out = x.new_empty((T * topk, width), dtype=torch.uint8), x.new_empty(size, dtype=torch.uint8)
    q, s = out
    _call("mx_dispatch_quantize", dev, p, T, K, _ld(x), _packed(slot_row, "dispatch_quantize: slot_row must be int32", torch.int32, T * topk, dev),
          topk, _packed(row_offsets, "dispatch_quantize: row_offsets must be int32", torch.int32, E + 1, dev), E, MX_FORMAT[fmt],
          _packed(q, "dispatch_quantize: q", torch.uint8, T * topk * width, dev), _packed(s, "dispatch_quantize: s", torch.uint8, size, dev))
    return q, s


def combine(rows: torch.Tensor, slot_row: torch.Tensor, weights=None, out_dtype=None, out=None):
    """mx_combine: y[t] = sum_j weights[t, j] * rows[slot_row[t, j]] (weights None: all 1), in fp32, rounded once to
    out_dtype (rows' type if None). Slots with a negative slot_row have no part. With weights=None it is also the
    gradient of an unquantized dispatch."""
    p = _matrix(rows, "combine: rows must be a 2-D fp32 or BF16 CUDA tensor with unit column stride", _FLOATS)
    _need(slot_row.dim() == 2, "combine: slot_row [T, topk]")
    (T, topk), N, dev = slot_row.shape, rows.shape[1], rows.device
    if out is None:
        out = rows.new_empty((T, N), dtype=out_dtype or rows.dtype)
    _call("mx_combine", dev, p, _out_code(rows.dtype), rows.shape[0], _ld(rows),
          _packed(slot_row, "combine: slot_row must be int32", torch.int32, T * topk, dev),
          None if weights is None else _packed(weights, "combine: weights must be fp32 [T, topk]", torch.float32, T * topk, dev),
          T, topk, N, _matrix(out, "combine: out", _FLOATS, (T, N), dev), _out_code(out.dtype), _ld(out))
    return out


def combine_backward(dy: torch.Tensor, rows: torch.Tensor, slot_row: torch.Tensor, weights=None, need_weights: bool = True, out=None):
    """mx_combine_bwd: (d_rows like rows, d_weights fp32 [T, topk]) from dy [T, N]. need_weights=False leaves
    d_weights out (None), and rows is then only asked for its shape and type. Padding rows get zeros. No two slots may
    name the same row."""
    p = _matrix(rows, "combine_backward: rows must be a 2-D fp32 or BF16 CUDA tensor with unit column stride", _FLOATS)
    _need(slot_row.dim() == 2, "combine_backward: slot_row [T, topk]")
    (T, topk), (R, N), dev = slot_row.shape, rows.shape, rows.device
    if out is None:
        # Every row of a plan's partition is written; rows that no slot names stay as they are, so they start as 0.
        out = (rows.new_empty((R, N)) if R == T * topk else rows.new_zeros((R, N)),
               rows.new_empty((T, topk), dtype=torch.float32) if need_weights else None)
    d_rows, d_weights = out
    _call("mx_combine_bwd", dev, _matrix(dy, "combine_backward: dy must be [T, N], fp32 or BF16", _FLOATS, (T, N), dev), _out_code(dy.dtype), _ld(dy),
          p, _out_code(rows.dtype), R, _ld(rows), _packed(slot_row, "combine_backward: slot_row must be int32", torch.int32, T * topk, dev),
          None if weights is None else _packed(weights, "combine_backward: weights must be fp32 [T, topk]", torch.float32, T * topk, dev),
          T, topk, N, _matrix(d_rows, "combine_backward: d_rows", (rows.dtype,), (R, N), dev), _ld(d_rows),
          None if d_weights is None else _packed(d_weights, "combine_backward: d_weights", torch.float32, T * topk, dev))
    return d_rows, d_weights


def grid_equal(a: torch.Tensor, b: torch.Tensor, out=None):
    """mx_grid_equal over the bytes of two CUDA tensors. Returns (mismatches, first_index) as
    1-element int64 device tensors (no host synchronisation)."""
    assert a.is_contiguous() and b.is_contiguous()
    n = a.numel() * a.element_size()
    assert b.numel() * b.element_size() == n
    if out is None:
        out = torch.empty(2, dtype=torch.int64, device=a.device)
    cnt, first = out[0:1], out[1:2]
    st = lib().mx_grid_equal(_p(a), _p(b), n, _p(cnt), _p(first), ctypes.c_void_p(_stream(a.device)))
    _check(st, "mx_grid_equal")
    return cnt, first


def device_error() -> int:
    """Reads and clears the device status word (synchronizes). 0 means no error bit set."""
    bits = ctypes.c_uint32(0)
    st = lib().mx_device_error(ctypes.byref(bits))
    if st not in (0, -6):
        _check(st, "mx_device_error")
    return int(bits.value)


def set_wait_timeout_ns(ns: int):
    lib().mx_set_wait_timeout_ns(int(ns))


GEMM_PAIR, GEMM_SINGLE = 0, 1


def set_gemm_variant(variant: int):
    """0: CTA-pair GEMM kernel (default); 1: single-CTA kernel."""
    lib().mx_set_gemm_variant(int(variant))


QUANT_REGISTERS, QUANT_TMA, QUANT_SPLIT = 0, 1, 2


def set_quantize_variant(variant: int):
    """0: register-staged quantizer (default; split loads for long rowwise tile walks); 1: TMA-staged
    quantizer; 2: register-staged with split loads for every rowwise call. Same bytes in every case."""
    lib().mx_set_quantize_variant(int(variant))
