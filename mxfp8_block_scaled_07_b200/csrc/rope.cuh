// Rotary positions: pairs of a head's features turned by an angle that grows with the token's position.
//
// Pair i of a head at position p:  y_a = x_a c - x_b s,  y_b = x_b c + x_a s  with (c, s) = (cos, sin)[p, i] from a
// table in fp32 (which carries any stretching for long contexts, and a factor on both). Pairs are (i, i + rot / 2) in
// the half layout and (2i, 2i + 1) in the interleaved one; features from rot on are copied. The gradient is the same
// with -s. Each sum of two products is formed as fma(x_a, c, -w) + fma(-x_b, s, w), w = x_b s rounded (Kahan's difference
// of products, within 1.5 ulp however much cancels), so that one rounding to the output type is all that is lost.
//
// Bound by HBM: an element is read and written once; a thread keeps its pairs' cosines and sines in registers over
// several heads of a token, so that the table adds a few percent. 12 288 tokens of 40 heads of 128 in BF16 take 44 us each way
// (5.8 TB/s), 5201 of 12 heads of 128 in fp32, half rotated, 14.5 us (4.5 TB/s); 13 tokens of 32 heads 1.8 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fastdiv.cuh"
#include "ptx.cuh"

namespace mx {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;

// a c - b s. An infinite b s leaves w - b s undefined; the infinity itself is then the answer.
__device__ __forceinline__ float diff_of_products(float a, float c, float b, float s) {
    const float w = b * s;
    const float e = fmaf(-b, s, w), f = fmaf(a, c, -w);
    return e == e ? f + e : f;
}

// ---- table -------------------------------------------------------------------------------------------------

struct RopeTableArgs {
    double freq[kRopeMaxPairs];
    float* table;            // [count, 2 n]: cosines, then sines
    double amplitude;
    int64_t first, count;
    FastDiv n;               // pairs
};

// Angles, cosines and sines in fp64, rounded once: at position 10^6 an fp32 angle would be off by 0.03.
__global__ void __launch_bounds__(kRopeThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
    grid_wait();
    const int n = static_cast<int>(a.n.d);
    for (int64_t p = blockIdx.x; p < a.count; p += gridDim.x) {
        const double at = static_cast<double>(a.first + p);
        for (int i = threadIdx.x; i < n; i += kRopeThreads) {
            double sn, cs;
            sincos(at * a.freq[i], &sn, &cs);
            a.table[p * 2 * n + i] = static_cast<float>(a.amplitude * cs);
            a.table[p * 2 * n + n + i] = static_cast<float>(a.amplitude * sn);
        }
    }
}

// ---- elements ----------------------------------------------------------------------------------------------

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }

// V elements: one 16-byte access where V of them fill one, else one by one.
template <class T, int V>
struct Piece {
    static constexpr bool kWide = V * sizeof(T) == 16;
    union {
        uint4 w;
        T e[V];
    };
    __device__ Piece() {}
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kWide) {
            w = ld_once_v4(p);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kWide) {
            *reinterpret_cast<uint4*>(p) = w;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = e[i];
        }
    }
};

// n consecutive fp32 table entries (16-byte accesses where n is a multiple of 4: the caller's rows are then aligned).
template <int N>
__device__ __forceinline__ void load_angles(const float* p, float (&out)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            out[i] = v.x, out[i + 1] = v.y, out[i + 2] = v.z, out[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = p[i];
    }
}

struct RopeArgs {
    const void* x;
    void* y;
    const float* table;         // [positions, rot]
    const void* pos;            // int32 or int64 [T], or null: 0 .. T - 1
    int64_t ldx_t, ldx_h, ldy_t, ldy_h;
    int64_t positions, T;
    FastDiv lanes, chunks;      // pieces of a head; head chunks of a token
    uint32_t* err;
    int H, D, rot, pair_lanes;
    int pos64, negate, copy;    // copy: features from rot on are written too (y is not x)
};

// Zeros in a thread's pieces of its heads; in place, where no thread has the features from rot on, those that turn the others share them.
template <class T, int V, bool IL>
__device__ __noinline__ void zero_heads(const RopeArgs& a, T* y, int chunk, int step, int piece) {
    Piece<T, V> none;
#pragma unroll
    for (int i = 0; i < V; ++i) none.e[i] = from_f32<T>(0.0f);
    auto zeros = [&](T* p, int d, int end) {
        if (d + V <= end) none.store(p + d);
        else
            for (int e = d; e < end; ++e) p[e] = from_f32<T>(0.0f);
    };
    for (int h = chunk; h < a.H; h += step) {
        T* p = y + h * a.ldy_h;
        if (piece >= a.pair_lanes) {
            zeros(p, a.rot + (piece - a.pair_lanes) * V, a.D);
            continue;
        }
        zeros(p, piece * V, a.rot);
        if (!IL) zeros(p, a.rot / 2 + piece * V, a.rot);
        if (!a.copy)
            for (int d = a.rot + piece * V; d < a.D; d += a.pair_lanes * V) zeros(p, d, a.D);
    }
}

// One thread: one piece of every head of a chunk (heads chunk, chunk + chunks, ...: the threads of a token walk
// neighbouring heads together), V elements of both halves in the half layout, V consecutive ones in the interleaved.
// HC heads are loaded before the first is written. A negative position is a padding token: zeros. A position behind
// the table: zeros, and the device status word says so.
template <class T, int V, bool IL, int HC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    grid_wait();
    constexpr int W = IL ? V / 2 : V;              // pairs per piece
    const uint32_t gid = blockIdx.x * kRopeThreads + threadIdx.x;
    const uint32_t unit = a.lanes.div(gid);
    const int piece = static_cast<int>(gid - unit * a.lanes.d);
    const uint32_t t = a.chunks.div(unit);
    const int chunk = static_cast<int>(unit - t * a.chunks.d), step = static_cast<int>(a.chunks.d);
    if (t >= a.T) return;
    const T* x = static_cast<const T*>(a.x) + t * a.ldx_t;
    T* y = static_cast<T*>(a.y) + t * a.ldy_t;
    int64_t p = t;
    if (a.pos) p = a.pos64 ? static_cast<const int64_t*>(a.pos)[t] : static_cast<const int32_t*>(a.pos)[t];
    const bool known = p >= 0 && p < a.positions;
    if (p >= a.positions) atomicOr(a.err, kErrBadIndex);
    if (!known) {                                  // every thread zeros of its own
        zero_heads<T, V, IL>(a, y, chunk, step, piece);
        return;
    }
    if (piece >= a.pair_lanes) {                   // features that are not rotated
        const int d = a.rot + (piece - a.pair_lanes) * V;
        const bool whole = d + V <= a.D;
        for (int h0 = chunk; h0 < a.H; h0 += HC * step) {
            Piece<T, V> v[HC];
#pragma unroll
            for (int j = 0; j < HC; ++j) {
                const int h = h0 + j * step;
                if (h < a.H && whole) v[j].load(x + h * a.ldx_h + d);
            }
#pragma unroll
            for (int j = 0; j < HC; ++j) {
                const int h = h0 + j * step;
                if (h >= a.H) break;
                if (whole) {
                    v[j].store(y + h * a.ldy_h + d);
                } else {
                    for (int e = d; e < a.D; ++e) y[h * a.ldy_h + e] = x[h * a.ldx_h + e];
                }
            }
        }
        return;
    }
    float c[W], s[W];
    load_angles<W>(a.table + p * a.rot + piece * W, c);
    load_angles<W>(a.table + p * a.rot + a.rot / 2 + piece * W, s);
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = a.negate ? -s[i] : s[i];
    const int d0 = piece * V, d1 = a.rot / 2 + piece * V;
    for (int h0 = chunk; h0 < a.H; h0 += HC * step) {
        Piece<T, V> u[HC], w[IL ? 1 : HC];
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            const int h = h0 + j * step;
            if (h < a.H) {
                u[j].load(x + h * a.ldx_h + d0);
                if constexpr (!IL) w[j].load(x + h * a.ldx_h + d1);
            }
        }
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            const int h = h0 + j * step;
            if (h >= a.H) break;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                T& ta = IL ? u[j].e[2 * i] : u[j].e[i];
                T& tb = IL ? u[j].e[(2 * i + 1) % V] : w[IL ? 0 : j].e[i];
                const float xa = to_f32(ta), xb = to_f32(tb);
                ta = from_f32<T>(diff_of_products(xa, c[i], xb, s[i]));
                tb = from_f32<T>(diff_of_products(xb, c[i], -xa, s[i]));
            }
            u[j].store(y + h * a.ldy_h + d0);
            if constexpr (!IL) w[j].store(y + h * a.ldy_h + d1);
        }
    }
}

}  // namespace mx
