// A paged cache of keys and values in E4M3 with one E8M0 scale per page and head, and tokens appended to it.
//
// Codes [pages, heads, page, D] (a page's tokens of one head are consecutive: page x D bytes), scale bytes [pages,
// heads]. The grid is the library's (OCP MX v1.0) with the block made of a page's tokens of one head: e = floor(log2 amax) - 8,
// code = RNE(x 2^-e) saturated to +-448. A page that tokens are appended to over several calls keeps e from falling:
// when the new tokens need a larger one the page's other codes are rounded anew to it, which a power of two makes exact but for
// codes that become subnormal. A page with NaN or infinity has scale byte 0xFF and zero codes until it is begun anew.
//
// Keys are rotated on the way, and their codes are those of the exact rotation. A sum of two products within 1.5 ulp has the exact one's
// code unless it lies next to a tie between codes or a power of two; those sums (one in 2^16) are formed in fp64
// and rounded to odd, which rounds to E4M3 as the exact value does.
//
// One token of 64 sequences, 8 key and 32 query heads of 128: 2.6 us, a chain of four loads. Prompts of 10 200 tokens: queries 31 us
// (5.3 TB/s), keys and values 35 us, 73% of the issue slots busy with the rotation, its check and the codes.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "quantize.cuh"
#include "rope.cuh"

namespace mx {

// a c - b s rounded to odd in fp32 (towards zero, and the last bit set unless exact), a and b of 8 bits: rounding that to at most 22
// bits gives what rounding the exact value would. In fp64, where a c is exact and one rounding is left, made in each direction. (Beyond
// fp32's range: an infinity.)
__device__ __forceinline__ float diff_to_odd(float a, float c, float b, float s) {
    const float near = __fmaf_rn(a, c, -__fmul_rn(b, s));
    // No number; a pair that is not turned (the first position), which is exact.
    if (!(fabsf(near) < INFINITY) || (c == 1.0f && s == 0.0f)) return near;
    const double p = static_cast<double>(a) * c, x = -static_cast<double>(b), y = s;
    const float f = __double2float_rz(__fma_rz(x, y, p));
    return __fma_rd(x, y, p) == f && __fma_ru(x, y, p) == f ? f : __int_as_float(__float_as_int(f) | 1);
}

// a c - b s within 1.5 ulp (rope.cuh), and whether a rounding to E4M3 under any power of two, or the power of two below, may hang on
// what is missing: ties between codes have 5 bits, so the last 19 bits of a number within 1.5 ulp of one are within 4 units of zero
// (3 below a power of two). Below 2^-100, where products lose bits, always; but 0 is exact, or less than 2^-147 and its code 0.
__device__ __forceinline__ float diff_in_doubt(float a, float c, float b, float s, bool& doubt) {
    const float w = __fmul_rn(b, s), y = __fsub_rn(__fmaf_rn(a, c, -w), __fmaf_rn(b, s, -w));      // keeps the sign of zeros
    doubt = (((__float_as_uint(y) + 4) & 0x7FFFF) <= 8 || fabsf(y) < 0x1p-100f) && y != 0.0f;
    return y;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 2^(s - 127) of a scale byte below 255.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s ? s << 23 : 1u << 22); }
// Scale byte from the largest magnitude (fp32 bits without the sign) of a block: max(E - 8, 0), 0xFF for NaN or Inf.
__device__ __forceinline__ uint32_t scale_byte_of(uint32_t amax_bits) {
    const int E = static_cast<int>(amax_bits >> 23);
    return E == 255 ? 255u : static_cast<uint32_t>(max(E - 8, 0));
}
__device__ __forceinline__ float inv_scale_of(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Two values to two E4M3 codes (the first in the low byte).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two E4M3 codes (16 bits) to f16x2, exactly.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3_hi(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// Four codes rounded anew after a factor (a power of two below 1).
__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float f) {
    const uint32_t a = f16x2_of_e4m3(codes), b = f16x2_of_e4m3_hi(codes);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return e4m3x2(x.x * f, x.y * f) | (e4m3x2(y.x * f, y.y * f) << 16);
}

struct CacheView {
    uint8_t *k, *v;               // codes; a page's [heads, page, D] block is packed
    uint8_t *ks, *vs;             // scale bytes; a page's [heads] are packed
    int64_t k_page, v_page, ks_page, vs_page;      // bytes from one page to the next
    const int32_t* table;         // page ids [B, width], row stride ld_table
    int64_t ld_table;
    const int32_t* lengths;       // [B]
    const int32_t* row_offsets;   // [B + 1], or null: one row per sequence
    int64_t pages;
    int32_t width, B, T, Hkv, page_shift;
};

// Rows [first, first + n) of the batch are sequence b's, whatever the offsets hold: inside [0, T).
__device__ __forceinline__ void rows_of(const CacheView& c, int b, int& first, int& n) {
    if (!c.row_offsets) {
        first = b, n = 1;
        return;
    }
    first = min(max(c.row_offsets[b], 0), c.T);
    n = min(max(c.row_offsets[b + 1] - first, 0), c.T - first);
}

// Page id of a sequence's page, or -1 outside the table or the pool.
__device__ __forceinline__ int64_t page_id(const CacheView& c, int b, int64_t index) {
    if (index >= c.width) return -1;
    const int32_t id = c.table[b * c.ld_table + index];
    return id < 0 || id >= c.pages ? -1 : id;
}

struct AppendArgs {
    CacheView c;
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16* q_out;
    const float* table;           // rotations [positions, rot], or null: none
    int64_t ldk_t, ldk_h, ldv_t, ldv_h, ldq_t, ldq_h, ldo_t, ldo_h;
    int64_t positions;
    uint32_t* err;
    int Hq, D, rot, interleaved;
    int kv_blocks;                // append_one_kernel: blocks that append; the ones behind them rotate queries
    FastDiv heads2;               // 2 * Hkv
};

// Elements [d, d + 8) of a row, rotated, and a bit for each that is in doubt. x: the row's head.
__device__ __forceinline__ uint32_t rotated8(const __nv_bfloat16* x, int d, const float* angles, int rot, bool interleaved, float (&y)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(x + d);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) y[2 * i] = bf16_lo(u[i]), y[2 * i + 1] = bf16_hi(u[i]);
    if (d >= rot) return 0;
    const int h = rot / 2;
    uint32_t doubts = 0;
    bool doubt;
    if (interleaved) {
        float c[4], s[4];
        load_angles<4>(angles + d / 2, c);
        load_angles<4>(angles + h + d / 2, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = diff_in_doubt(a, c[i], b, s[i], doubt);
            doubts |= doubt ? 1u << 2 * i : 0u;
            y[2 * i + 1] = diff_in_doubt(b, c[i], -a, s[i], doubt);
            doubts |= doubt ? 2u << 2 * i : 0u;
        }
        return doubts;
    }
    const bool low = d < h;
    const int i0 = low ? d : d - h;
    const uint4 o = *reinterpret_cast<const uint4*>(x + (low ? d + h : d - h));
    const uint32_t v[4] = {o.x, o.y, o.z, o.w};
    float c[8], s[8];
    load_angles<8>(angles + i0, c);
    load_angles<8>(angles + h + i0, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = i & 1 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
        y[i] = diff_in_doubt(y[i], c[i], low ? other : -other, s[i], doubt);
        doubts |= doubt ? 1u << i : 0u;
    }
    return doubts;
}
// Element d of a row again, without doubt.
__device__ __forceinline__ float rotated_to_odd(const __nv_bfloat16* x, int d, const float* angles, int rot, bool interleaved) {
    const int h = rot / 2;
    const bool first = interleaved ? !(d & 1) : d < h;
    const int other = interleaved ? d ^ 1 : first ? d + h : d - h, pair = interleaved ? d / 2 : first ? d : d - h;
    const float b = to_f32(x[other]);
    return diff_to_odd(to_f32(x[d]), angles[pair], first ? b : -b, angles[h + pair]);
}

// The angles of a position: null where there is no rotation, `bad` where the position lies outside the table.
__device__ __forceinline__ const float* angles_of(const AppendArgs& a, int64_t pos, bool& bad) {
    bad = a.table && (pos < 0 || pos >= a.positions);
    if (bad && pos >= 0) atomicOr(a.err, kErrBadIndex);
    return a.table && !bad ? a.table + pos * a.rot : nullptr;
}

// A sequence with its rows [first, first + n) and its length.
struct Found {
    int b, first, n;
    int64_t len;
};
// The last sequence whose key(first row, number) is at most `x` (keys rise with the sequence), by a whole warp; b < 0: none. A lane
// per sequence, with all that is asked of it loaded at once: the search costs one round trip for every 32 sequences.
template <class Key>
__device__ __forceinline__ Found find_sequence(const CacheView& c, int x, Key key) {
    Found f{-1, 0, 0, 0};
    for (int b0 = 0; b0 < c.B; b0 += 32) {
        const int b = min(b0 + static_cast<int>(threadIdx.x & 31), c.B - 1);
        int first, n;
        rows_of(c, b, first, n);
        const int len = c.lengths[b];
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, b0 + static_cast<int>(threadIdx.x & 31) < c.B && key(first, b) <= x)) - 1;
        if (at < 0) break;
        f = {b0 + at, __shfl_sync(0xFFFFFFFFu, first, at), __shfl_sync(0xFFFFFFFFu, n, at), __shfl_sync(0xFFFFFFFFu, len, at)};
        if (at < 31) break;
    }
    return f;
}

// One row of queries by THREADS threads (`tid` of them; whole warps). A thread keeps the angles of its piece (eight pairs, or
// eight features that are copied) over the heads that it walks, HC of them on their way at a time. Rows that no sequence
// holds are left alone.
template <int THREADS, int HC>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int row, int tid) {
    const CacheView& c = a.c;
    const Found q = c.row_offsets ? find_sequence(c, row, [](int first, int) { return first; }) : Found{row, row, 1, c.lengths[row]};
    if (q.b < 0 || row < q.first || row >= q.first + q.n) return;
    const int64_t pos = q.len - q.n + (row - q.first);
    bool bad;
    const float* angles = angles_of(a, pos, bad);
    bad |= pos < 0;
    const int rot = angles ? a.rot : 0, half = a.rot / 2;
    const int pairs = a.interleaved ? rot / 8 : rot / 16;  // pieces that are rotated; the others are copied
    const int lanes = pairs + (a.D - rot) / 8;
    const int slots = THREADS / lanes, slot = tid / lanes, piece = tid - slot * lanes;
    if (slot >= slots) return;
    const __nv_bfloat16* x = a.q + row * a.ldq_t;
    __nv_bfloat16* y = a.q_out + row * a.ldo_t;
    const bool turn = piece < pairs, two = turn && !a.interleaved;
    const int d0 = turn ? piece * 8 : rot + (piece - pairs) * 8;
    float cs[8], sn[8];
    if (turn && two) {
        load_angles<8>(angles + d0, cs);
        load_angles<8>(angles + half + d0, sn);
    } else if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = angles[d0 / 2 + i], sn[i] = angles[half + d0 / 2 + i];
    }
    for (int h0 = slot; h0 < a.Hq; h0 += HC * slots) {
        Piece<__nv_bfloat16, 8> u[HC], w[HC];
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            const int h = h0 + j * slots;
            u[j].w = w[j].w = make_uint4(0, 0, 0, 0);
            if (h < a.Hq && !bad) {
                u[j].load(x + h * a.ldq_h + d0);
                if (two) w[j].load(x + h * a.ldq_h + half + d0);
            }
        }
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            const int h = h0 + j * slots;
            if (h >= a.Hq) break;
            if (two) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = to_f32(u[j].e[i]), q = to_f32(w[j].e[i]);
                    u[j].e[i] = from_f32<__nv_bfloat16>(diff_of_products(p, cs[i], q, sn[i]));
                    w[j].e[i] = from_f32<__nv_bfloat16>(diff_of_products(q, cs[i], -p, sn[i]));
                }
                w[j].store(y + h * a.ldo_h + half + d0);
            } else if (turn) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = to_f32(u[j].e[2 * i]), q = to_f32(u[j].e[2 * i + 1]);
                    u[j].e[2 * i] = from_f32<__nv_bfloat16>(diff_of_products(p, cs[i], q, sn[i]));
                    u[j].e[2 * i + 1] = from_f32<__nv_bfloat16>(diff_of_products(q, cs[i], -p, sn[i]));
                }
            }
            u[j].store(y + h * a.ldo_h + d0);
        }
    }
}

__device__ __forceinline__ uint32_t amax_bits8(const float (&y)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    return m;
}
__device__ __forceinline__ uint2 encode8(const float (&y)[8], float inv) {
    return make_uint2(e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16),
                      e4m3x2(y[4] * inv, y[5] * inv) | (e4m3x2(y[6] * inv, y[7] * inv) << 16));
}

constexpr int kAppendOneThreads = 128;

// One new token per sequence: a warp per (sequence, head, keys or values), D / 8 lanes of eight elements.
template <int D>
__global__ void __launch_bounds__(kAppendOneThreads) append_one_kernel(const __grid_constant__ AppendArgs a) {
    grid_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CacheView& c = a.c;
    if (static_cast<int>(blockIdx.x) >= a.kv_blocks) {
        rotate_queries<kAppendOneThreads, 2>(a, blockIdx.x - a.kv_blocks, threadIdx.x);
        return;
    }
    const uint32_t item = blockIdx.x * (kAppendOneThreads / 32) + warp;
    const int b = a.heads2.div(item), r = item - b * a.heads2.d, h = r >> 1;
    if (b >= c.B) return;
    const bool keys = !(r & 1);
    const int64_t pos = static_cast<int64_t>(c.lengths[b]) - 1;
    if (pos < 0) return;
    const int slot = static_cast<int>(pos & ((1 << c.page_shift) - 1));
    const int64_t id = page_id(c, b, pos >> c.page_shift);
    if (id < 0) {
        if (lane == 0) atomicOr(a.err, kErrBadIndex);
        return;
    }
    uint8_t* codes = (keys ? c.k + id * c.k_page : c.v + id * c.v_page) + (static_cast<int64_t>(h) << c.page_shift) * D;
    uint8_t* scale = (keys ? c.ks + id * c.ks_page : c.vs + id * c.vs_page) + h;
    const uint32_t was = slot ? *scale : 0u;
    float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (lane < D / 8) {
        if (keys) {
            bool bad;
            const float* angles = angles_of(a, pos, bad);
            const __nv_bfloat16* x = a.k + b * a.ldk_t + h * a.ldk_h;
            uint32_t doubts = bad ? 0 : rotated8(x, lane * 8, angles, angles ? a.rot : 0, a.interleaved, y);
#pragma unroll 1
            for (; doubts; doubts &= doubts - 1) {
                const int i = __ffs(doubts) - 1;
                const float exact = rotated_to_odd(x, lane * 8 + i, angles, a.rot, a.interleaved);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = k == i ? exact : y[k];
            }
        } else {
            rotated8(a.v + b * a.ldv_t + h * a.ldv_h, lane * 8, nullptr, 0, false, y);
        }
    }
    const uint32_t s = max(was, scale_byte_of(__reduce_max_sync(0xFFFFFFFFu, amax_bits8(y))));
    if (s > was && slot) {                       // the page's other codes, 16 at a time
        const float f = s == 255 ? 0.0f : scale_value(was) * inv_scale_of(s);
        for (int i = lane; i < (D / 16) << c.page_shift; i += 32) {
            if (i / (D / 16) == slot) continue;
            uint4 w = *reinterpret_cast<const uint4*>(codes + i * 16);
            w = s == 255 ? make_uint4(0, 0, 0, 0) : make_uint4(rescaled(w.x, f), rescaled(w.y, f), rescaled(w.z, f), rescaled(w.w, f));
            *reinterpret_cast<uint4*>(codes + i * 16) = w;
        }
    }
    if (lane < D / 8)
        *reinterpret_cast<uint2*>(codes + slot * D + lane * 8) = s == 255 ? make_uint2(0, 0) : encode8(y, inv_scale_of(s));
    if (lane == 0) *scale = static_cast<uint8_t>(s);
}

// The queries of prompts: a warp per row. A kernel of its own, since it needs half the registers of the one below and lives
// on many rows on their way (together, with a block per row, 10 200 tokens of 32 + 8 heads took 107 us).
constexpr int kAppendQueryThreads = 256;
__global__ void __launch_bounds__(kAppendQueryThreads) append_queries_kernel(const __grid_constant__ AppendArgs a) {
    grid_wait();
    const int row = blockIdx.x * (kAppendQueryThreads / 32) + (threadIdx.x >> 5);
    if (row < a.c.T) rotate_queries<32, 4>(a, row, threadIdx.x & 31);
}

// Any number of new tokens per sequence: a block per (page of a sequence, head, keys or values), CH pieces of eight
// elements per thread (page x D = 8 CH threads). What bounds it is the chain of loads from the offsets to the keys: two pieces a thread
// leave most warps on their way (eight a thread took 60 us for 10 200 tokens of 8 heads; forming every sum exactly in fp32 instead of those in
// doubt 39). Blocks are numbered without a prefix sum: sequence b's pages start at
// floor(row_offsets[b] / page) + 2 b, which leaves room for all that its tokens can touch (n tokens touch at most n / page +
// 2 pages); blocks for which nothing is left return.
template <int D, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 1024 ? 1 : 1536 / THREADS) append_kernel(const __grid_constant__ AppendArgs a) {
    grid_wait();
    __shared__ uint32_t warp_max[THREADS / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CacheView& c = a.c;
    const int item = a.heads2.div(blockIdx.x), r = blockIdx.x - item * a.heads2.d, h = r >> 1;
    const bool keys = !(r & 1);
    const int ps = c.page_shift, page = 1 << ps;
    const Found q = find_sequence(c, item, [&](int first, int b) { return (first >> ps) + 2 * b; });
    if (q.b < 0) return;
    const int first = q.first, n = q.n;
    const int64_t len = q.len, start = len - n;
    const int nth = item - ((first >> ps) + 2 * q.b);
    const int64_t index = (max(start, int64_t(0)) >> ps) + nth;
    const int64_t base = index << ps;            // position of the page's first token
    if (n <= 0 || nth < 0 || base >= len) return;
    const int lo = static_cast<int>(max(start - base, int64_t(0))), hi = static_cast<int>(min(len - base, int64_t(page)));
    const int64_t id = page_id(c, q.b, index);   // on its way with the tokens
    float y[CH][8];
    uint32_t m = 0, doubts = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int at = i * THREADS + threadIdx.x, tok = at / (D / 8), d = (at % (D / 8)) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = 0.0f;
        if (tok >= lo && tok < hi) {
            const int64_t row = first + (base + tok - start);
            if (keys) {
                bool bad;
                const float* angles = angles_of(a, base + tok, bad);
                if (!bad) doubts |= rotated8(a.k + row * a.ldk_t + h * a.ldk_h, d, angles, angles ? a.rot : 0, a.interleaved, y[i]) << 8 * i;
            } else {
                rotated8(a.v + row * a.ldv_t + h * a.ldv_h, d, nullptr, 0, false, y[i]);
            }
        }
    }
    // Elements in doubt (one in 2^16; one in 8 of what is not turned) from memory, one by one: with their inputs kept for that, the
    // kernel spilled.
#pragma unroll 1
    for (; doubts; doubts &= doubts - 1) {
        const int k = __ffs(doubts) - 1, at = k / 8 * THREADS + threadIdx.x, tok = at / (D / 8), d = (at % (D / 8)) * 8 + k % 8;
        const float exact = rotated_to_odd(a.k + (first + (base + tok - start)) * a.ldk_t + h * a.ldk_h, d, a.table + (base + tok) * a.rot, a.rot, a.interleaved);
#pragma unroll
        for (int i = 0; i < 8 * CH; ++i) y[i / 8][i % 8] = i == k ? exact : y[i / 8][i % 8];
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) m = max(m, amax_bits8(y[i]));
    if (id < 0) {                                    // the same in the whole block
        if (threadIdx.x == 0) atomicOr(a.err, kErrBadIndex);
        return;
    }
    uint8_t* codes = (keys ? c.k + id * c.k_page : c.v + id * c.v_page) + (static_cast<int64_t>(h) << ps) * D;
    uint8_t* scale = (keys ? c.ks + id * c.ks_page : c.vs + id * c.vs_page) + h;
    const uint32_t was = lo ? *scale : 0u;           // before the barrier, behind which it is written
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) warp_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) m = max(m, warp_max[w]);
    const uint32_t s = max(was, scale_byte_of(m));
    const float inv = s == 255 ? 0.0f : inv_scale_of(s), f = s == 255 ? 0.0f : scale_value(was) * inv;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int at = i * THREADS + threadIdx.x, tok = at / (D / 8);
        uint2* p = reinterpret_cast<uint2*>(codes + at * 8);
        if (tok >= lo && tok < hi) {
            *p = s == 255 ? make_uint2(0, 0) : encode8(y[i], inv);
        } else if (lo > 0 && s > was) {
            const uint2 w = *p;
            *p = s == 255 ? make_uint2(0, 0) : make_uint2(rescaled(w.x, f), rescaled(w.y, f));
        }
    }
    if (threadIdx.x == 0) *scale = static_cast<uint8_t>(s);
}

}  // namespace mx
