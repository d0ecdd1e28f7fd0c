// Tokens into the experts' rows and back: dispatch with quantization, combine, and combine's gradient.
//
// Between the router and the grouped expert GEMMs ("End-to-End MXFP8 Reinforcement Learning on
// Blackwell", Table 2: 20 480 tokens, top-8 of 128 experts, 163 840 rows): slot (t, j) of token t lives
// in row slot_row[t, j] of the experts' operand; a slot without an expert holds ~row, a padding row.
//   dispatch:         q[row(t, j)], scales = quantize(x[t])      (zeros in padding rows)
//   combine:          y[t] = sum_j w[t, j] c[row(t, j)]
//   combine backward: dc[row(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], c[row(t, j)]>
// All three walk tokens, not rows: a token is read (and quantized) once and its k rows are written, or
// its k rows are read and it is written, so nothing is moved twice and no sum needs atomics. Each is
// bound by HBM; loads and stores are whole 16- or 32-byte pieces of consecutive lanes.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "fp4.cuh"
#include "quantize.cuh"
#include "route.cuh"

namespace mx {

constexpr int kExThreads = 256;

struct DispatchArgs {
    const uint16_t* x;        // BF16 [T, K], row stride ldx
    const int32_t* slot_row;  // [T, k]
    const int32_t* offsets;   // [E + 1]
    uint8_t* q;               // [T * k, K] E4M3 or [T * k, K / 2] packed E2M1
    uint8_t* s;               // grouped tensor-core layout, `tiles` 128-row tiles of ctiles blocks
    int64_t T, K, ldx, n;     // n = T * k rows
    int64_t units;            // T * chunks warp units, then `tiles` units for the layout's pads
    int k, E, chunks, ctiles, kblocks, tiles;
    int vec32;                // x rows and q 32-byte aligned: 256-bit accesses
};

// First 128-row tile of the scale layout of every group, from the row offsets (shared memory, by the
// whole CTA). Returns nothing; first[E] is the number of tiles in use.
__device__ __forceinline__ void expert_tiles(const int32_t* offsets, int E, int32_t* off, int32_t* first,
                                             int32_t* warp_sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e <= E; e += kExThreads) off[e] = offsets[e];
    __syncthreads();
    const int per = (E + kExThreads - 1) / kExThreads;       // consecutive groups per thread
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < E) sum += (max(off[e + 1] - off[e], 0) + 127) / 128;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < E) {
            first[e] = at;
            at += (max(off[e + 1] - off[e], 0) + 127) / 128;
            if (e == E - 1) first[E] = at;
        }
    }
    __syncthreads();
}

// Largest e in [0, E) with a[e] <= x (a nondecreasing).
__device__ __forceinline__ int last_not_above(const int32_t* a, int E, int x) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One warp unit = one token and 1024 of its columns: lane l quantizes 32-block l of the piece once and
// writes its codes to the token's k rows (32 or 16 bytes per lane, consecutive over the warp); four
// lanes join their scale bytes into one 4-byte word of the grouped layout, which L2 merges into whole
// sectors. Further units zero the layout's pads: the rows behind each group's last in its last 128-row
// tile, and the tiles behind the last group.
template <bool FP4>
__global__ void __launch_bounds__(kExThreads) dispatch_kernel(const __grid_constant__ DispatchArgs a) {
    __shared__ int32_t off[kRouteMaxExperts + 1];
    __shared__ int32_t first[kRouteMaxExperts + 1];
    __shared__ int32_t warp_sums[kExThreads / 32];
    expert_tiles(a.offsets, a.E, off, first, warp_sums);
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kExThreads / 32);
    const int64_t row_bytes = FP4 ? a.K / 2 : a.K;
    const int64_t tok_units = a.T * a.chunks;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kExThreads / 32) + (threadIdx.x >> 5); u < a.units;
         u += nwarps) {
        if (u >= tok_units) {
            const int tile = static_cast<int>(u - tok_units);
            int valid = 0;
            if (tile < first[a.E]) {
                const int e = last_not_above(first, a.E, tile);
                valid = min(128, off[e + 1] - off[e] - (tile - first[e]) * 128);
            }
            if (valid < 128) {
                uint8_t* base = a.s + static_cast<int64_t>(tile) * a.ctiles * 512 + lane * 16;
                for (int c = 0; c < a.ctiles; ++c, base += 512)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (lane + 32 * j >= valid) *reinterpret_cast<uint32_t*>(base + 4 * j) = 0;
            }
            continue;
        }
        const int64_t t = u / a.chunks;
        const int kb = static_cast<int>(u % a.chunks) * 32 + lane;
        const bool in = kb < a.kblocks;
        Block32 b;
        b.v[0] = b.v[1] = b.v[2] = b.v[3] = make_uint4(0, 0, 0, 0);
        if (in) {
            const uint16_t* p = a.x + t * a.ldx + static_cast<int64_t>(kb) * 32;
            if (a.vec32) {
                ld_stream_v8(p, b.v[0], b.v[1]);
                ld_stream_v8(p + 16, b.v[2], b.v[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) b.v[j] = ld_cached_v4(p + 8 * j);
            }
        }
        const uint32_t amax = block_absmax(b);
        uint32_t sc;
        uint4 o0, o1;
        if constexpr (FP4) {
            sc = fp4_scale_byte(amax);
            o0 = fp4_encode_block(b, sc);
        } else {
            sc = scale_byte_from_amax(amax);
            uint2 e;
            e = encode_chunk(b.v[0], sc);
            o0.x = e.x; o0.y = e.y;
            e = encode_chunk(b.v[1], sc);
            o0.z = e.x; o0.w = e.y;
            e = encode_chunk(b.v[2], sc);
            o1.x = e.x; o1.y = e.y;
            e = encode_chunk(b.v[3], sc);
            o1.z = e.x; o1.w = e.y;
        }
        // The four K-blocks of a scale word sit in four neighbouring lanes.
        uint32_t word = (in ? sc : 0u) << (8 * (lane & 3));
        word |= __shfl_xor_sync(kFullMask, word, 1);
        word |= __shfl_xor_sync(kFullMask, word, 2);
        for (int j0 = 0; j0 < a.k; j0 += 32) {
            int row = -1, srow = 0, pad = 0;
            if (j0 + lane < a.k) {
                row = a.slot_row[t * a.k + j0 + lane];
                pad = row < 0;
                if (pad) row = ~row;
                if (row < a.n) {
                    const int e = last_not_above(off, a.E, row);
                    srow = first[e] * 128 + row - off[e];
                    if (srow < 0 || srow >= a.tiles * 128) row = -1;     // offsets that are no partition
                } else {
                    row = -1;
                }
            }
            const int m = min(32, a.k - j0);
            for (int j = 0; j < m; ++j) {
                const int64_t r = __shfl_sync(kFullMask, row, j);
                const int64_t sr = __shfl_sync(kFullMask, srow, j);
                const bool z = __shfl_sync(kFullMask, pad, j) != 0;
                if (r < 0) continue;
                if (in) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    uint8_t* q = a.q + r * row_bytes + static_cast<int64_t>(kb) * (FP4 ? 16 : 32);
                    if constexpr (FP4) {
                        *reinterpret_cast<uint4*>(q) = z ? zero : o0;
                    } else if (a.vec32) {
                        st_v8(q, z ? zero : o0, z ? zero : o1);
                    } else {
                        reinterpret_cast<uint4*>(q)[0] = z ? zero : o0;
                        reinterpret_cast<uint4*>(q)[1] = z ? zero : o1;
                    }
                }
                if ((lane & 3) == 0 && (kb >> 2) < a.ctiles) {
                    const int64_t blk = (sr >> 7) * a.ctiles + (kb >> 2);
                    *reinterpret_cast<uint32_t*>(a.s + blk * 512 + (sr & 31) * 16 + ((sr & 127) >> 5) * 4) = z ? 0u : word;
                }
            }
        }
    }
}

// ---- combine ----------------------------------------------------------------------------------------

struct CombineArgs {
    const void* c;            // [rows, N], row stride ldc
    const int32_t* slot_row;  // [T, k]
    const float* w;           // [T, k] or null (all 1)
    void* y;                  // [T, N], row stride ldy
    int64_t T, N, ldc, ldy, rows;
    int k, chunks;
    int vec;                  // 16-byte aligned rows: vector accesses
    // backward
    const void* dy;           // [T, N], row stride lddy
    void* dc;                 // [rows, N], row stride lddc, or null
    float* dw;                // [T, k] or null
    int64_t lddy, lddc;
};

// Eight consecutive columns per lane: 16 bytes of BF16, 32 of fp32.
template <class ELT>
__device__ __forceinline__ void load8(const ELT* p, float (&f)[8]) {
    if constexpr (sizeof(ELT) == 2) {
        const uint4 v = ld_stream_v4(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const uint4 v0 = ld_stream_v4(p), v1 = ld_stream_v4(p + 4);
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
}

template <class ELT>
__device__ __forceinline__ void store8(ELT* p, const float (&f)[8]) {
    if constexpr (sizeof(ELT) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

__device__ __forceinline__ float elt_to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float elt_to_float(float v) { return v; }
__device__ __forceinline__ void float_to_elt(float f, uint16_t& o) { o = __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ void float_to_elt(float f, float& o) { o = f; }

// A lane's eight columns of the 256-column piece that starts at column c0: consecutive ones with vector
// accesses, else every 32nd (element accesses stay coalesced). Entries past N read 0.
template <class ELT>
__device__ __forceinline__ void load_piece(const ELT* row, int64_t c0, int64_t N, int lane, bool vec, float (&f)[8]) {
    if (vec) {
        const int64_t c = c0 + lane * 8;
        if (c + 8 <= N) {
            load8(row + c, f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = c + i < N ? elt_to_float(row[c + i]) : 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = c0 + lane + 32 * i;
            f[i] = c < N ? elt_to_float(row[c]) : 0.0f;
        }
    }
}

template <class ELT>
__device__ __forceinline__ void store_piece(ELT* row, int64_t c0, int64_t N, int lane, bool vec, const float (&f)[8]) {
    if (vec && c0 + lane * 8 + 8 <= N) {
        store8(row + c0 + lane * 8, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = vec ? c0 + lane * 8 + i : c0 + lane + 32 * i;
            if (c < N) float_to_elt(f[i], row[c]);
        }
    }
}

// One warp per (token, 256 columns): the k rows' pieces are loaded four at a time, so that four
// independent loads are in flight per lane, and added in slot order in fp32; one rounding at the end.
template <class CT, class YT>
__global__ void __launch_bounds__(kExThreads) combine_kernel(const __grid_constant__ CombineArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t u = static_cast<int64_t>(blockIdx.x) * (kExThreads / 32) + (threadIdx.x >> 5);
    if (u >= a.T * a.chunks) return;
    const int64_t t = u / a.chunks, c0 = (u % a.chunks) * 256;
    const CT* c = static_cast<const CT*>(a.c);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        float f[4][8], w[4];
        int64_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = -1;
            w[j] = 1.0f;
            if (j0 + j < a.k) {
                r[j] = a.slot_row[t * a.k + j0 + j];
                if (r[j] >= a.rows) r[j] = -1;
                if (a.w) w[j] = a.w[t * a.k + j0 + j];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r[j] >= 0) load_piece(c + r[j] * a.ldc, c0, a.N, lane, a.vec != 0, f[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r[j] >= 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], f[j][i], acc[i]);
            }
    }
    store_piece(static_cast<YT*>(a.y) + t * a.ldy, c0, a.N, lane, a.vec != 0, acc);
}

// One block per token: warp w takes the 256-column pieces w, w + 8, ...; per piece dy is loaded once and
// each of the token's rows is read (for dw) and written (dc). Each warp's dot products are joined through
// shared memory in warp order, so dw does not depend on timing. Four slots per pass keep the row pieces
// in registers; a further pass re-reads dy, which L1 or L2 holds.
template <class CT, class YT>
__global__ void __launch_bounds__(kExThreads) combine_bwd_kernel(const __grid_constant__ CombineArgs a) {
    __shared__ float part[kExThreads / 32][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const CT* c = static_cast<const CT*>(a.c);
    const YT* dy = static_cast<const YT*>(a.dy) + t * a.lddy;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        int64_t r[4];
        bool pad[4];
        float w[4], dot[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = -1;
            pad[j] = false;
            w[j] = 1.0f;
            if (j0 + j < a.k) {
                const int s = a.slot_row[t * a.k + j0 + j];
                pad[j] = s < 0;
                r[j] = pad[j] ? ~s : s;
                if (r[j] >= a.rows) r[j] = -1;
                if (a.w) w[j] = a.w[t * a.k + j0 + j];
            }
        }
        for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.N; c0 += kExThreads * 8) {
            float g[8], f[4][8];
            load_piece(dy, c0, a.N, lane, a.vec != 0, g);
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r[j] >= 0 && !pad[j]) load_piece(c + r[j] * a.ldc, c0, a.N, lane, a.vec != 0, f[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r[j] >= 0 && !pad[j]) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[j][i], dot[j]);
                    }
            }
            if (a.dc) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r[j] >= 0) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = pad[j] ? 0.0f : w[j] * g[i];
                        store_piece(static_cast<CT*>(a.dc) + r[j] * a.lddc, c0, a.N, lane, a.vec != 0, o);
                    }
            }
        }
        if (a.dw) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dot[j] = warp_sum(dot[j]);
                if (lane == 0) part[warp][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < 4 && j0 + static_cast<int>(threadIdx.x) < a.k) {
                float s = 0.0f;
#pragma unroll
                for (int v = 0; v < kExThreads / 32; ++v) s += part[v][threadIdx.x];
                a.dw[t * a.k + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

}  // namespace mx
