// The call path of the binding's MXFP4 and expert-routing functions: checks of the tensors, allocation of the outputs
// and the library call (include/mx.h), in one native function per entry point.
//
// What a small call costs is host time: through Python attribute checks, torch.empty and ctypes a call took 11 to 15 us
// for a kernel of 2 to 5 us. Nothing else happens here: sizes and flags are checked by the library, and every function
// returns after its launches, on the current stream of the tensors' device, with that device current.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/mx.h"

// The torch and the Python this was built for, for build.py and mx.py to read from the file before it is loaded.
extern "C" __attribute__((used, visibility("default"))) const char mx_call_tag[] = "mx-call-tag:" MX_CALL_TAG ";";

namespace {

PyObject* g_error = nullptr;       // the binding's MxError(status, what)

struct Refused {
    int status;
    std::string what;
};

void need(bool ok, const char* what) {
    if (!ok) throw Refused{MX_ERR_ARG, what};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    need(THPVariable_Check(o), what);
    return THPVariable_Unpack(o);
}
const at::Tensor* optional_tensor(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);       // takes anything with __index__
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

constexpr int kF32 = 1, kBf16 = 2, kU8 = 4;

bool type_in(const at::Tensor& t, int types) {
    switch (t.scalar_type()) {
        case at::kFloat: return types & kF32;
        case at::kBFloat16: return types & kBf16;
        case at::kByte: return types & kU8;
        default: return false;
    }
}
mx_out_dtype code_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? MX_OUT_BF16 : MX_OUT_F32; }
at::ScalarType type_of(int64_t code) { return code == MX_OUT_BF16 ? at::kBFloat16 : at::kFloat; }

// A 2-D CUDA tensor with unit column stride. Of a single row no stride is ever used: its own width stands for it.
struct Matrix {
    void* p;
    int64_t m, n, ld;
};
Matrix matrix(const at::Tensor& t, int types, const char* what) {
    need(t.is_cuda() && t.dim() == 2 && type_in(t, types) && (t.stride(1) == 1 || t.size(1) <= 1), what);
    return {t.data_ptr(), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1)};
}
Matrix matrix(const at::Tensor& t, int types, int64_t m, int64_t n, at::Device dev, const char* what) {
    const Matrix x = matrix(t, types, what);
    need(x.m == m && x.n == n && t.device() == dev, what);
    return x;
}

// A contiguous tensor of `numel` elements on `dev`.
void* packed(const at::Tensor& t, at::ScalarType type, int64_t numel, at::Device dev, const char* what) {
    need(t.scalar_type() == type && t.numel() == numel && t.is_contiguous() && t.device() == dev, what);
    return t.data_ptr();
}

// An uninitialized tensor on the current device (Place has made the tensors' device current), from the caching allocator as
// at::empty gives it, without the dispatcher.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) {
    return at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), type,
                                     std::nullopt);
}

template <class T>
T* ptr(void* p) {
    return static_cast<T*>(p);
}

// The tensors' device made current for the call, and its current stream.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    mx_stream stream;
    explicit Place(const at::Tensor& t) {
        need(t.is_cuda(), "CUDA tensors");
        if (t.device().index() != c10::cuda::current_device()) guard.set_device(t.device());
        stream = reinterpret_cast<mx_stream>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
    }
};

void check(mx_status st, const char* name) {
    if (st != MX_OK) throw Refused{st, name};
}

int64_t layout_bytes(int64_t rows, int64_t kblocks) { return (rows + 127) / 128 * 128 * ((kblocks + 3) / 4 * 4); }

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* tuple(std::initializer_list<PyObject*> items) {
    PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}
// Entry i of the caller's `out` tuple; its values stay the caller's own tensors in what is returned.
PyObject* out_item(PyObject* out, Py_ssize_t i, Py_ssize_t n, const char* what) {
    need(PyTuple_Check(out) && PyTuple_GET_SIZE(out) == n, what);
    return PyTuple_GET_ITEM(out, i);
}
PyObject* same(PyObject* o) {
    Py_INCREF(o);
    return o;
}

using Args = PyObject* const*;

// (logits, topk, score, bias, groups, topk_groups, group_score, renormalize, scale, out)
PyObject* route(Args a) {
    const at::Tensor& logits = tensor(a[0], "route: logits");
    const Matrix x = matrix(logits, kF32 | kBf16, "route: logits must be a 2-D fp32 or BF16 CUDA tensor with unit column stride");
    const at::Device dev = logits.device();
    const int64_t topk = integer(a[1]), score = integer(a[2]), groups = integer(a[4]), tg = integer(a[5]);
    const int64_t gs = integer(a[6]);
    const bool renorm = truth(a[7]);
    const float scale = static_cast<float>(number(a[8]));
    const at::Tensor* bias = optional_tensor(a[3], "route: bias");
    const void* pb = bias ? packed(*bias, at::kFloat, x.n, dev, "route: bias must be fp32 [E]") : nullptr;
    need(topk >= 1 && topk <= x.n, "route: 1 <= topk <= experts");      // before outputs of that width are allocated
    const Place place(logits);
    at::Tensor ids, weights;
    PyObject *oi = nullptr, *ow = nullptr;
    if (a[9] == Py_None) {
        ids = fresh({x.m, topk}, at::kInt);
        weights = fresh({x.m, topk}, at::kFloat);
    } else {
        oi = out_item(a[9], 0, 2, "route: out (ids, weights)");
        ow = out_item(a[9], 1, 2, "route: out (ids, weights)");
        ids = tensor(oi, "route: ids");
        weights = tensor(ow, "route: weights");
    }
    void* pi = packed(ids, at::kInt, x.m * topk, dev, "route: ids must be int32 [T, topk]");
    void* pw = packed(weights, at::kFloat, x.m * topk, dev, "route: weights must be fp32 [T, topk]");
    check(mx_route(x.p, code_of(logits), x.m, x.n, x.ld, ptr<const float>(const_cast<void*>(pb)), static_cast<int>(score),
                   groups, tg, static_cast<int>(gs), topk, renorm, scale, ptr<int32_t>(pi), ptr<float>(pw), place.stream),
          "mx_route");
    return tuple({oi ? same(oi) : wrap(ids), ow ? same(ow) : wrap(weights)});
}

// (d_weights, logits, ids, score, renormalize, scale, out)
PyObject* route_backward(Args a) {
    const at::Tensor &dw = tensor(a[0], "route_backward: d_weights"), &logits = tensor(a[1], "route_backward: logits");
    const at::Tensor& ids = tensor(a[2], "route_backward: ids");
    const Matrix x = matrix(logits, kF32 | kBf16, "route_backward: logits must be a 2-D fp32 or BF16 CUDA tensor with unit column stride");
    const at::Device dev = logits.device();
    need(ids.dim() == 2, "route_backward: ids [T, topk]");
    const int64_t topk = ids.size(1), score = integer(a[3]);
    const bool renorm = truth(a[4]);
    const float scale = static_cast<float>(number(a[5]));
    const void* pd = packed(dw, at::kFloat, x.m * topk, dev, "route_backward: d_weights must be fp32 [T, topk]");
    const void* pi = packed(ids, at::kInt, x.m * topk, dev, "route_backward: ids must be int32 [T, topk]");
    const Place place(logits);
    const at::Tensor out = a[6] == Py_None ? fresh({x.m, x.n}, logits.scalar_type()) : tensor(a[6], "route_backward: out");
    const Matrix o = matrix(out, code_of(logits) == MX_OUT_BF16 ? kBf16 : kF32, x.m, x.n, dev, "route_backward: out must be like logits");
    check(mx_route_bwd(static_cast<const float*>(pd), x.p, code_of(logits), x.m, x.n, x.ld, static_cast<const int32_t*>(pi),
                       static_cast<int>(score), topk, renorm, scale, o.p, o.ld, place.stream),
          "mx_route_bwd");
    return a[6] == Py_None ? wrap(out) : same(a[6]);
}

// (ids, experts, out)
PyObject* route_plan(Args a) {
    const at::Tensor& ids = tensor(a[0], "route_plan: ids must be an int32 CUDA tensor");
    const at::Device dev = ids.device();
    const int64_t n = ids.numel(), experts = integer(a[1]);
    const void* pi = packed(ids, at::kInt, n, dev, "route_plan: ids must be a contiguous int32 tensor");
    const int64_t bytes = mx_route_plan_workspace_bytes(n, experts);
    need(bytes >= 0, "route_plan: 1 to 1024 experts");
    const Place place(ids);
    at::Tensor off, slot_row, counts, ws;
    PyObject* o[3] = {nullptr, nullptr, nullptr};
    if (a[2] == Py_None) {
        off = fresh({experts + 1}, at::kInt);
        slot_row = fresh(ids.sizes(), at::kInt);
        counts = fresh({experts}, at::kInt);
    } else {
        for (int i = 0; i < 3; ++i) o[i] = out_item(a[2], i, 3, "route_plan: out (row_offsets, slot_row, counts)");
        off = tensor(o[0], "route_plan: row_offsets");
        slot_row = tensor(o[1], "route_plan: slot_row");
        counts = tensor(o[2], "route_plan: counts");
    }
    if (bytes) ws = fresh({bytes}, at::kByte);
    void* po = packed(off, at::kInt, experts + 1, dev, "route_plan: row_offsets must be int32 [experts + 1]");
    void* ps = packed(slot_row, at::kInt, n, dev, "route_plan: slot_row must be int32 like ids");
    void* pc = packed(counts, at::kInt, experts, dev, "route_plan: counts must be int32 [experts]");
    check(mx_route_plan(static_cast<const int32_t*>(pi), n, experts, ptr<int32_t>(po), ptr<int32_t>(ps), ptr<int32_t>(pc),
                        bytes ? ws.data_ptr() : nullptr, place.stream),
          "mx_route_plan");
    return tuple({o[0] ? same(o[0]) : wrap(off), o[1] ? same(o[1]) : wrap(slot_row), o[2] ? same(o[2]) : wrap(counts)});
}

// (x, slot_row, row_offsets, format, out)
PyObject* dispatch_quantize(Args a) {
    const at::Tensor &x = tensor(a[0], "dispatch_quantize: x"), &slot_row = tensor(a[1], "dispatch_quantize: slot_row");
    const at::Tensor& off = tensor(a[2], "dispatch_quantize: row_offsets");
    const Matrix m = matrix(x, kBf16, "dispatch_quantize: x must be a 2-D BF16 CUDA tensor with unit column stride");
    need(slot_row.dim() == 2 && slot_row.size(0) == m.m && off.numel() >= 2, "dispatch_quantize: slot_row [T, topk], row_offsets [E + 1]");
    const at::Device dev = x.device();
    const int64_t topk = slot_row.size(1), E = off.numel() - 1, fmt = integer(a[3]);
    const int64_t rows = m.m * topk, width = fmt == MX_FORMAT_E2M1 ? m.n / 2 : m.n;
    const int64_t size = (rows + 127 * std::min(E, rows)) / 128 * 128 * ((m.n / 32 + 3) / 4 * 4);
    const void* ps = packed(slot_row, at::kInt, rows, dev, "dispatch_quantize: slot_row must be int32");
    const void* po = packed(off, at::kInt, E + 1, dev, "dispatch_quantize: row_offsets must be int32");
    const Place place(x);
    at::Tensor q, s;
    PyObject *oq = nullptr, *os = nullptr;
    if (a[4] == Py_None) {
        q = fresh({rows, width}, at::kByte);
        s = fresh({size}, at::kByte);
    } else {
        oq = out_item(a[4], 0, 2, "dispatch_quantize: out (q, s)");
        os = out_item(a[4], 1, 2, "dispatch_quantize: out (q, s)");
        q = tensor(oq, "dispatch_quantize: q");
        s = tensor(os, "dispatch_quantize: s");
    }
    void* pq = packed(q, at::kByte, rows * width, dev, "dispatch_quantize: q");
    void* pl = packed(s, at::kByte, size, dev, "dispatch_quantize: s");
    check(mx_dispatch_quantize(m.p, m.m, m.n, m.ld, static_cast<const int32_t*>(ps), topk, static_cast<const int32_t*>(po), E,
                               static_cast<mx_format>(fmt), ptr<uint8_t>(pq), ptr<uint8_t>(pl), place.stream),
          "mx_dispatch_quantize");
    return tuple({oq ? same(oq) : wrap(q), os ? same(os) : wrap(s)});
}

// (rows, slot_row, weights, out type code or -1 for rows' own, out)
PyObject* combine(Args a) {
    const at::Tensor &rows = tensor(a[0], "combine: rows"), &slot_row = tensor(a[1], "combine: slot_row");
    const Matrix c = matrix(rows, kF32 | kBf16, "combine: rows must be a 2-D fp32 or BF16 CUDA tensor with unit column stride");
    need(slot_row.dim() == 2, "combine: slot_row [T, topk]");
    const at::Device dev = rows.device();
    const int64_t T = slot_row.size(0), topk = slot_row.size(1), code = integer(a[3]);
    const void* ps = packed(slot_row, at::kInt, T * topk, dev, "combine: slot_row must be int32");
    const at::Tensor* w = optional_tensor(a[2], "combine: weights");
    const void* pw = w ? packed(*w, at::kFloat, T * topk, dev, "combine: weights must be fp32 [T, topk]") : nullptr;
    const Place place(rows);
    const at::Tensor out = a[4] == Py_None ? fresh({T, c.n}, code < 0 ? rows.scalar_type() : type_of(code)) : tensor(a[4], "combine: out");
    const Matrix y = matrix(out, kF32 | kBf16, T, c.n, dev, "combine: out must be [T, N], fp32 or BF16");
    check(mx_combine(c.p, code_of(rows), c.m, c.ld, static_cast<const int32_t*>(ps), static_cast<const float*>(pw), T, topk, c.n, y.p,
                     code_of(out), y.ld, place.stream),
          "mx_combine");
    return a[4] == Py_None ? wrap(out) : same(a[4]);
}

// (dy, rows, slot_row, weights, need_weights, out)
PyObject* combine_backward(Args a) {
    const at::Tensor &dy = tensor(a[0], "combine_backward: dy"), &rows = tensor(a[1], "combine_backward: rows");
    const at::Tensor& slot_row = tensor(a[2], "combine_backward: slot_row");
    const Matrix c = matrix(rows, kF32 | kBf16, "combine_backward: rows must be a 2-D fp32 or BF16 CUDA tensor with unit column stride");
    need(slot_row.dim() == 2, "combine_backward: slot_row [T, topk]");
    const at::Device dev = rows.device();
    const int64_t T = slot_row.size(0), topk = slot_row.size(1);
    const bool need_weights = truth(a[4]);
    const Matrix d = matrix(dy, kF32 | kBf16, T, c.n, dev, "combine_backward: dy must be [T, N], fp32 or BF16");
    const void* ps = packed(slot_row, at::kInt, T * topk, dev, "combine_backward: slot_row must be int32");
    const at::Tensor* w = optional_tensor(a[3], "combine_backward: weights");
    const void* pw = w ? packed(*w, at::kFloat, T * topk, dev, "combine_backward: weights must be fp32 [T, topk]") : nullptr;
    const Place place(rows);
    at::Tensor d_rows, d_w;
    PyObject *orow = nullptr, *ow = nullptr;
    bool weights_out = need_weights;
    if (a[5] == Py_None) {
        d_rows = fresh({c.m, c.n}, rows.scalar_type());
        // Every row of a plan's partition is written; rows that no slot names stay as they are, so they start as 0.
        if (c.m != T * topk) d_rows.zero_();
        if (need_weights) d_w = fresh({T, topk}, at::kFloat);
    } else {
        orow = out_item(a[5], 0, 2, "combine_backward: out (d_rows, d_weights)");
        ow = out_item(a[5], 1, 2, "combine_backward: out (d_rows, d_weights)");
        d_rows = tensor(orow, "combine_backward: d_rows");
        weights_out = ow != Py_None;
        if (weights_out) d_w = tensor(ow, "combine_backward: d_weights");
    }
    const Matrix o = matrix(d_rows, code_of(rows) == MX_OUT_BF16 ? kBf16 : kF32, c.m, c.n, dev, "combine_backward: d_rows must be like rows");
    float* pdw = weights_out ? ptr<float>(packed(d_w, at::kFloat, T * topk, dev, "combine_backward: d_weights must be fp32 [T, topk]")) : nullptr;
    check(mx_combine_bwd(d.p, code_of(dy), d.ld, c.p, code_of(rows), c.m, c.ld, static_cast<const int32_t*>(ps),
                         static_cast<const float*>(pw), T, topk, c.n, o.p, o.ld, pdw, place.stream),
          "mx_combine_bwd");
    return tuple({orow ? same(orow) : wrap(d_rows), ow ? same(ow) : (need_weights ? wrap(d_w) : same(Py_None))});
}

// (x, flags, out)
PyObject* quantize_fp4(Args a) {
    const at::Tensor& x = tensor(a[0], "quantize_fp4: x");
    const Matrix m = matrix(x, kBf16, "quantize_fp4: x must be a 2-D BF16 CUDA tensor with unit column stride");
    const int64_t flags = integer(a[1]);
    const bool row = flags & MX_ROWWISE, col = flags & MX_COLWISE, swz = flags & MX_SWIZZLE;
    if (m.n % 32 != 0 || (col && m.m % 32 != 0)) throw Refused{MX_ERR_SHAPE, "quantize_fp4: blocks of 32 along the quantized axis"};
    const at::Device dev = x.device();
    const Place place(x);
    const bool want[4] = {row, row, col, col};
    const int64_t bytes[4] = {m.m * m.n / 2, swz ? layout_bytes(m.m, m.n / 32) : m.m * (m.n / 32), m.m * m.n / 2,
                              swz ? layout_bytes(m.n, m.m / 32) : m.n * (m.m / 32)};
    const int64_t shape[4][2] = {{m.m, m.n / 2}, {m.m, m.n / 32}, {m.n, m.m / 2}, {m.n, m.m / 32}};
    at::Tensor t[4];
    void* p[4] = {nullptr, nullptr, nullptr, nullptr};
    for (int i = 0; i < 4; ++i) {
        if (!want[i]) continue;
        if (a[2] != Py_None) {
            t[i] = tensor(out_item(a[2], i, 4, "quantize_fp4: out (q_row, s_row, q_col, s_col)"), "quantize_fp4: out");
            p[i] = packed(t[i], at::kByte, bytes[i], dev, "quantize_fp4: out (q_row, s_row, q_col, s_col)");
        } else {
            t[i] = (i & 1) && swz ? fresh({bytes[i]}, at::kByte) : fresh({shape[i][0], shape[i][1]}, at::kByte);
            p[i] = t[i].data_ptr();
        }
    }
    check(mx_quantize_fp4(m.p, m.m, m.n, m.ld, static_cast<int>(flags), ptr<uint8_t>(p[0]), ptr<uint8_t>(p[1]), ptr<uint8_t>(p[2]),
                          ptr<uint8_t>(p[3]), place.stream),
          "mx_quantize_fp4");
    if (a[2] != Py_None) return same(a[2]);
    PyObject* r[4];
    for (int i = 0; i < 4; ++i) r[i] = want[i] ? wrap(t[i]) : same(Py_None);
    return tuple({r[0], r[1], r[2], r[3]});
}

// (q, s, swizzled, out)
PyObject* dequantize_fp4(Args a) {
    const at::Tensor &q = tensor(a[0], "dequantize_fp4: q"), &s = tensor(a[1], "dequantize_fp4: s");
    const bool swz = truth(a[2]);
    need(q.is_cuda() && q.dim() == 2, "dequantize_fp4: q must be a 2-D uint8 CUDA tensor");
    const at::Device dev = q.device();
    const int64_t M = q.size(0), K = 2 * q.size(1);
    const void* pq = packed(q, at::kByte, M * K / 2, dev, "dequantize_fp4: q must be contiguous uint8");
    const void* ps = packed(s, at::kByte, swz ? layout_bytes(M, K / 32) : M * (K / 32), dev, "dequantize_fp4: s");
    const Place place(q);
    const at::Tensor out = a[3] == Py_None ? fresh({M, K}, at::kBFloat16) : tensor(a[3], "dequantize_fp4: out");
    const Matrix o = matrix(out, kBf16, M, K, dev, "dequantize_fp4: out must be BF16 [M, K]");
    check(mx_dequantize_fp4(static_cast<const uint8_t*>(pq), static_cast<const uint8_t*>(ps), M, K, swz, o.p, o.ld, place.stream),
          "mx_dequantize_fp4");
    return a[3] == Py_None ? wrap(out) : same(a[3]);
}

// (qa, sa, qb, sb, out type code, out)
PyObject* gemm_fp4(Args a) {
    const at::Tensor &qa = tensor(a[0], "gemm_fp4: qa"), &sa = tensor(a[1], "gemm_fp4: sa_swz");
    const at::Tensor &qb = tensor(a[2], "gemm_fp4: qb"), &sb = tensor(a[3], "gemm_fp4: sb_swz");
    need(qa.is_cuda() && qa.dim() == 2 && qb.dim() == 2 && qa.size(1) == qb.size(1), "gemm_fp4: qa [M, K/2] and qb [N, K/2], uint8 CUDA tensors");
    const at::Device dev = qa.device();
    const int64_t M = qa.size(0), N = qb.size(0), K = 2 * qa.size(1);
    const void* pa = packed(qa, at::kByte, M * K / 2, dev, "gemm_fp4: qa");
    const void* pb = packed(qb, at::kByte, N * K / 2, dev, "gemm_fp4: qb");
    const void* psa = packed(sa, at::kByte, layout_bytes(M, K / 32), dev, "gemm_fp4: sa_swz");
    const void* psb = packed(sb, at::kByte, layout_bytes(N, K / 32), dev, "gemm_fp4: sb_swz");
    const Place place(qa);
    const at::Tensor out = a[5] == Py_None ? fresh({M, N}, type_of(integer(a[4]))) : tensor(a[5], "gemm_fp4: out");
    const Matrix c = matrix(out, kF32 | kBf16, M, N, dev, "gemm_fp4: out must be [M, N], fp32 or BF16");
    check(mx_gemm_fp4(static_cast<const uint8_t*>(pa), static_cast<const uint8_t*>(psa), static_cast<const uint8_t*>(pb),
                      static_cast<const uint8_t*>(psb), M, N, K, c.p, c.ld, code_of(out), place.stream),
          "mx_gemm_fp4");
    return a[5] == Py_None ? wrap(out) : same(a[5]);
}

// (qa, sa, qb, sb, row_offsets, out type code, out)
PyObject* grouped_gemm_fp4(Args a) {
    const at::Tensor &qa = tensor(a[0], "grouped_gemm_fp4: qa"), &sa = tensor(a[1], "grouped_gemm_fp4: sa_swz");
    const at::Tensor &qb = tensor(a[2], "grouped_gemm_fp4: qb"), &sb = tensor(a[3], "grouped_gemm_fp4: sb_swz");
    const at::Tensor& off = tensor(a[4], "grouped_gemm_fp4: row_offsets");
    need(qa.is_cuda() && qa.dim() == 2 && qb.dim() == 3 && qb.size(2) == qa.size(1),
         "grouped_gemm_fp4: qa [rows, K/2] and qb [G, N, K/2], uint8 CUDA tensors");
    const at::Device dev = qa.device();
    const int64_t rows = qa.size(0), K = 2 * qa.size(1), G = qb.size(0), N = qb.size(1);
    const void* pa = packed(qa, at::kByte, rows * K / 2, dev, "grouped_gemm_fp4: qa");
    const void* pb = packed(qb, at::kByte, G * N * K / 2, dev, "grouped_gemm_fp4: qb");
    need(sa.numel() >= layout_bytes(rows, K / 32), "grouped_gemm_fp4: sa_swz");
    const void* psa = packed(sa, at::kByte, sa.numel(), dev, "grouped_gemm_fp4: sa_swz");
    const void* psb = packed(sb, at::kByte, G * layout_bytes(N, K / 32), dev, "grouped_gemm_fp4: sb_swz");
    const void* po = packed(off, at::kInt, G + 1, dev, "grouped_gemm_fp4: row_offsets must be int32 [G + 1]");
    const Place place(qa);
    const at::Tensor out = a[6] == Py_None ? fresh({rows, N}, type_of(integer(a[5]))) : tensor(a[6], "grouped_gemm_fp4: out");
    const Matrix c = matrix(out, kF32 | kBf16, rows, N, dev, "grouped_gemm_fp4: out must be [rows, N], fp32 or BF16");
    check(mx_grouped_gemm_fp4(static_cast<const uint8_t*>(pa), static_cast<const uint8_t*>(psa), static_cast<const uint8_t*>(pb),
                              static_cast<const uint8_t*>(psb), static_cast<const int32_t*>(po), G, rows, N, K, c.p, c.ld,
                              code_of(out), place.stream),
          "mx_grouped_gemm_fp4");
    return a[6] == Py_None ? wrap(out) : same(a[6]);
}

// Argument count, refusals as MxError(status, what), and torch's and Python's own errors as they are.
template <PyObject* (*F)(Args), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (nargs != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", N, nargs);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        if (PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", r.status, r.what.c_str()) : nullptr) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_XDECREF(g_error);
    g_error = same(cls);
    Py_RETURN_NONE;
}

#define MX_METHOD(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<&f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MX_METHOD(route, 10),
                         MX_METHOD(route_backward, 7),
                         MX_METHOD(route_plan, 3),
                         MX_METHOD(dispatch_quantize, 5),
                         MX_METHOD(combine, 5),
                         MX_METHOD(combine_backward, 6),
                         MX_METHOD(quantize_fp4, 3),
                         MX_METHOD(dequantize_fp4, 4),
                         MX_METHOD(gemm_fp4, 6),
                         MX_METHOD(grouped_gemm_fp4, 7),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mxcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxcall() { return PyModule_Create(&module); }
