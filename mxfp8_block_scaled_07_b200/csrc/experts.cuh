// Tokens into the experts' rows and back: dispatch with quantization, combine, and combine's gradient.
//
// Between the router and the grouped expert GEMMs ("End-to-End MXFP8 Reinforcement Learning on
// Blackwell", Table 2: 20 480 tokens, top-8 of 128 experts, 163 840 rows): slot (t, j) of token t lives
// in row slot_row[t, j] of the experts' operand; a slot without an expert holds ~row, a padding row.
//   dispatch:         q[row(t, j)], scales = quantize(x[t])      (zeros in padding rows)
//   combine:          y[t] = sum_j w[t, j] c[row(t, j)]
//   combine backward: dc[row(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], c[row(t, j)]>
// All three walk tokens, not rows: a token is read (and quantized) once and its k rows are written, or
// its k rows are read and it is written, so nothing is moved twice and no sum needs atomics. Combine
// is bound by HBM (20 480 x 8 x 2048 BF16: 6.2 TB/s, backward 5.4), dispatch by its stores to eight places per token (4.8
// TB/s); loads and stores are whole 16- or 32-byte pieces of consecutive lanes.
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
    uint32_t tok_units, units;    // T * chunks warp units, then `tiles` units for the layout's pads
    FastDiv chunks;           // pieces of 1024 columns per token
    int k, E, ctiles, kblocks, tiles;
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
    grid_wait();
    __shared__ int32_t off[kRouteMaxExperts + 1];
    __shared__ int32_t first[kRouteMaxExperts + 1];
    __shared__ int32_t warp_sums[kExThreads / 32];
    expert_tiles(a.offsets, a.E, off, first, warp_sums);
    const int lane = threadIdx.x & 31;
    const uint32_t nwarps = gridDim.x * (kExThreads / 32);
    const int64_t row_bytes = FP4 ? a.K / 2 : a.K;
    for (uint32_t u = blockIdx.x * (kExThreads / 32) + (threadIdx.x >> 5); u < a.units; u += nwarps) {
        if (u >= a.tok_units) {
            const int tile = static_cast<int>(u - a.tok_units);
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
        const uint32_t tu = a.chunks.div(u);
        const int64_t t = tu;
        const int kb = static_cast<int>(u - tu * a.chunks.d) * 32 + lane;
        const bool in = kb < a.kblocks;
        Block32 b;
        b.v[0] = b.v[1] = b.v[2] = b.v[3] = make_uint4(0, 0, 0, 0);
        if (in) {
            const uint16_t* p = a.x + t * a.ldx + static_cast<int64_t>(kb) * 32;
            if (a.vec32) {
                ld_once_v8(p, b.v[0], b.v[1]);
                ld_once_v8(p + 16, b.v[2], b.v[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) b.v[j] = reinterpret_cast<const uint4*>(p)[j];
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
    uint32_t units;           // T * chunks, < 2^31
    FastDiv chunks;           // pieces of a row, 512 bytes of c each
    int k;
    int vec;                  // 16-byte aligned rows: vector accesses
    // backward
    const void* dy;           // [T, N], row stride lddy
    void* dc;                 // [rows, N], row stride lddc, or null
    float* dw;                // [T, k] or null
    int64_t lddy, lddc;
};

constexpr int kCombineSlots = 8;      // slots whose rows are in flight together

__device__ __forceinline__ float elt_to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float elt_to_float(float v) { return v; }
__device__ __forceinline__ void float_to_elt(float f, uint16_t& o) { o = __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ void float_to_elt(float f, float& o) { o = f; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A piece of a row is 32 lanes x P elements. With vector accesses a lane has P consecutive elements
// (c0 + P lane ..), else every 32nd (c0 + lane + 32 i), so that element accesses stay coalesced.
template <int P>
__device__ __forceinline__ int64_t piece_col(int64_t c0, int lane, int i, bool vec) {
    return vec ? c0 + lane * P + i : c0 + lane + 32 * i;
}

// A lane's part of a piece of c, as it lies in memory: 8 BF16 or 4 fp32 in 16 bytes. Entries past N are 0.
__device__ __forceinline__ uint4 load_raw(const uint16_t* row, int64_t c0, int64_t N, int lane, bool vec) {
    if (vec && c0 + lane * 8 + 8 <= N) return ld_once_v4(row + c0 + lane * 8);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t col = piece_col<8>(c0, lane, i, vec);
        if (col < N) w[i >> 1] |= static_cast<uint32_t>(row[col]) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_raw(const float* row, int64_t c0, int64_t N, int lane, bool vec) {
    if (vec && c0 + lane * 4 + 4 <= N) return ld_once_v4(row + c0 + lane * 4);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t col = piece_col<4>(c0, lane, i, vec);
        if (col < N) w[i] = __float_as_uint(row[col]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}

// P elements of a row in any of the two types.
template <int P, class ELT>
__device__ __forceinline__ void load_floats(const ELT* row, int64_t c0, int64_t N, int lane, bool vec, float (&f)[P]) {
    if constexpr (P * sizeof(ELT) == 16) {
        unpack(load_raw(row, c0, N, lane, vec), f);
    } else {
        if (vec && c0 + lane * P + P <= N) {
            const ELT* p = row + c0 + lane * P;
            if constexpr (sizeof(ELT) == 2) {               // 4 BF16
                const uint2 v = *reinterpret_cast<const uint2*>(p);
                f[0] = __uint_as_float(v.x << 16);
                f[1] = __uint_as_float(v.x & 0xFFFF0000u);
                f[2] = __uint_as_float(v.y << 16);
                f[3] = __uint_as_float(v.y & 0xFFFF0000u);
            } else {                                        // 8 fp32
                const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
                f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t col = piece_col<P>(c0, lane, i, vec);
                f[i] = col < N ? elt_to_float(row[col]) : 0.0f;
            }
        }
    }
}
template <int P, class ELT>
__device__ __forceinline__ void store_floats(ELT* row, int64_t c0, int64_t N, int lane, bool vec, const float (&f)[P]) {
    if (vec && c0 + lane * P + P <= N) {
        ELT* p = row + c0 + lane * P;
        if constexpr (sizeof(ELT) == 2 && P == 8) {
            st_global_v4(p, make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
        } else if constexpr (sizeof(ELT) == 2) {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
        } else {
#pragma unroll
            for (int q = 0; q < P / 4; ++q)
                st_global_v4(p + 4 * q, make_uint4(__float_as_uint(f[4 * q]), __float_as_uint(f[4 * q + 1]),
                                                   __float_as_uint(f[4 * q + 2]), __float_as_uint(f[4 * q + 3])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t col = piece_col<P>(c0, lane, i, vec);
            if (col < N) float_to_elt(f[i], row[col]);
        }
    }
}

// Slot j0 + lane of token t for lanes < min(8, k - j0): its row (negative: none) and weight.
__device__ __forceinline__ void load_slot(const CombineArgs& a, int64_t t, int j0, int lane, int& row, float& w) {
    row = -1;
    w = 1.0f;
    if (lane < kCombineSlots && j0 + lane < a.k) {
        row = a.slot_row[t * a.k + j0 + lane];
        if (a.w) w = a.w[t * a.k + j0 + lane];
    }
}

// One warp per (token, 512 bytes of a row), warps walking the pieces of consecutive tokens together. The
// pieces of up to 8 rows are loaded before any is used, and the next unit's slots before this unit's
// arithmetic, so a warp has 4 KB in flight nearly all the time; terms are added in slot order in fp32 and
// rounded once. 20 480 tokens x 8 rows x 2048 BF16: 122 us, 6.2 TB/s (four rows at a time, slots loaded one by
// one: 271 us). Three blocks per SM: 122 us; two (no register limit) 137, four 129.
template <class CT, class YT>
__global__ void __launch_bounds__(kExThreads, 3) combine_kernel(const __grid_constant__ CombineArgs a) {
    grid_wait();
    constexpr int P = 16 / static_cast<int>(sizeof(CT));
    const int lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * (kExThreads / 32);
    const CT* c = static_cast<const CT*>(a.c);
    uint32_t u = blockIdx.x * (kExThreads / 32) + (threadIdx.x >> 5);
    if (u >= a.units) return;
    int row;
    float w;
    load_slot(a, a.chunks.div(u), 0, lane, row, w);
    for (;;) {
        const uint32_t tu = a.chunks.div(u);
        const int64_t t = tu, c0 = static_cast<int64_t>(u - tu * a.chunks.d) * (32 * P);
        const uint32_t next = u + step;
        float acc[P];
#pragma unroll
        for (int i = 0; i < P; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kCombineSlots) {
            uint4 v[kCombineSlots];
            const uint32_t live = __ballot_sync(kFullMask, row >= 0 && row < a.rows);
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) {
                const int64_t r = __shfl_sync(kFullMask, row, j);
                if ((live >> j) & 1u) v[j] = load_raw(c + r * a.ldc, c0, a.N, lane, a.vec != 0);
            }
            const float wj = w;
            if (j0 + kCombineSlots < a.k)
                load_slot(a, t, j0 + kCombineSlots, lane, row, w);
            else if (next < a.units)
                load_slot(a, a.chunks.div(next), 0, lane, row, w);
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) {
                const float ww = __shfl_sync(kFullMask, wj, j);
                if ((live >> j) & 1u) {
                    float f[P];
                    unpack(v[j], f);
#pragma unroll
                    for (int i = 0; i < P; ++i) acc[i] = fmaf(ww, f[i], acc[i]);
                }
            }
        }
        store_floats<P>(static_cast<YT*>(a.y) + t * a.ldy, c0, a.N, lane, a.vec != 0, acc);
        if (next >= a.units) break;
        u = next;
    }
}

// W warps per token, 8 / W tokens per block at a time (W: as many as a row has pieces, at most 8): warp w of a token
// takes the row pieces w, w + W, ...; per piece dy and the token's rows are loaded together, then the rows' gradients are written. Each warp reduces its 8 dot products with 9
// shuffles (halving the values with the lanes) and joins them through shared memory in warp order, so dw does
// not depend on timing. (A whole block for rows of one piece: 12 462 tokens x 1 x 120 took 66 us.) The next token's slots are loaded before this token's arithmetic. 20 480 tokens x 8 rows
// x 2048 BF16: 263 us, 5.4 TB/s, nearly half of it writes (four slots per pass, two barriers each: 609 us). A form
// without tests for partial pieces, for rows of whole ones, has two thirds of the instructions and took 327 us at two,
// three and four blocks per SM, with plain or streaming stores, and with the dot products before or after them.
template <class CT, class YT, int W>
__global__ void __launch_bounds__(kExThreads, 3) combine_bwd_kernel(const __grid_constant__ CombineArgs a) {
    grid_wait();
    constexpr int P = 16 / static_cast<int>(sizeof(CT)), kTokens = kExThreads / 32 / W;
    __shared__ float part[2][kExThreads / 32][kCombineSlots];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, mate = (threadIdx.x >> 5) / W;   // token of the block
    const CT* c = static_cast<const CT*>(a.c);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kTokens;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + mate;
    if (t >= a.T) return;                       // all of the token's warps
    int row, flip = 0;
    float w;
    load_slot(a, t, 0, lane, row, w);
    for (; t < a.T; t += step) {
        const YT* dy = static_cast<const YT*>(a.dy) + t * a.lddy;
        for (int j0 = 0; j0 < a.k; j0 += kCombineSlots, flip ^= 1) {
            const int mine = row >= 0 ? row : ~row;                      // a padding row's gradient is 0
            const bool in = lane < kCombineSlots && j0 + lane < a.k && mine < a.rows;
            const uint32_t write = __ballot_sync(kFullMask, in), live = __ballot_sync(kFullMask, in && row >= 0);
            const float wj = w;
            if (j0 + kCombineSlots < a.k)
                load_slot(a, t, j0 + kCombineSlots, lane, row, w);
            else if (t + step < a.T)
                load_slot(a, t + step, 0, lane, row, w);
            float dot[kCombineSlots];
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) dot[j] = 0.0f;
            for (int64_t c0 = static_cast<int64_t>(warp) * (32 * P); c0 < a.N; c0 += W * 32 * P) {
                uint4 v[kCombineSlots];
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < kCombineSlots; ++j) {
                        const int64_t r = __shfl_sync(kFullMask, mine, j);
                        if ((live >> j) & 1u) v[j] = load_raw(c + r * a.ldc, c0, a.N, lane, a.vec != 0);
                    }
                }
                float g[P];
                load_floats<P>(dy, c0, a.N, lane, a.vec != 0, g);
                if (a.dc) {
#pragma unroll
                    for (int j = 0; j < kCombineSlots; ++j) {
                        const int64_t r = __shfl_sync(kFullMask, mine, j);
                        const float ww = __shfl_sync(kFullMask, wj, j);
                        if ((write >> j) & 1u) {
                            const bool pad = !((live >> j) & 1u);
                            float o[P];
#pragma unroll
                            for (int i = 0; i < P; ++i) o[i] = pad ? 0.0f : ww * g[i];
                            store_floats<P>(static_cast<CT*>(a.dc) + r * a.lddc, c0, a.N, lane, a.vec != 0, o);
                        }
                    }
                }
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < kCombineSlots; ++j)
                        if ((live >> j) & 1u) {
                            float f[P];
                            unpack(v[j], f);
#pragma unroll
                            for (int i = 0; i < P; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
                        }
                }
            }
            if (a.dw) {
                // Lanes with bit b of the lane set keep the upper half of the values, the others the lower.
#pragma unroll
                for (int h = kCombineSlots / 2, b = 16; h >= 1; h >>= 1, b >>= 1) {
                    const bool up = (lane & b) != 0;
#pragma unroll
                    for (int j = 0; j < h; ++j) {
                        const float give = up ? dot[j] : dot[j + h];
                        const float keep = up ? dot[j + h] : dot[j];
                        dot[j] = keep + __shfl_xor_sync(kFullMask, give, b);
                    }
                }
                dot[0] += __shfl_xor_sync(kFullMask, dot[0], 2);
                dot[0] += __shfl_xor_sync(kFullMask, dot[0], 1);
                // Value index: bits 4, 3, 2 of the lane.
                if constexpr (W == 1) {
                    if ((lane & 3) == 0 && j0 + (lane >> 2) < a.k) a.dw[t * a.k + j0 + (lane >> 2)] = dot[0];
                } else {
                    if ((lane & 3) == 0) part[flip][mate * W + warp][lane >> 2] = dot[0];
                    // The token's warps alone: tokens of a block do not wait for one another.
                    if constexpr (W == kExThreads / 32)
                        __syncthreads();
                    else
                        asm volatile("bar.sync %0, %1;" ::"r"(1 + mate), "n"(32 * W) : "memory");
                    if (warp == 0 && lane < kCombineSlots && j0 + lane < a.k) {
                        float s = 0.0f;
#pragma unroll
                        for (int v = 0; v < W; ++v) s += part[flip][mate * W + v][lane];
                        a.dw[t * a.k + j0 + lane] = s;
                    }
                }
            }
        }
    }
}

}  // namespace mx
