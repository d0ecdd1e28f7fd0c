// Expert routing: the choice of experts and their weights from router logits, its gradient, and the
// experts' row partition of a batch (what the grouped GEMMs take as row offsets).
//
// Table 2 of "End-to-End MXFP8 Reinforcement Learning on Blackwell" runs Qwen3-30B-A3B (128 experts,
// top-8); its expert GEMMs read rows grouped by expert, and these kernels make that grouping.
//
//   s_e   = softmax_e(x) or sigmoid(x_e), over the experts with x_e > -inf (NaN counts as -inf, +inf
//           as the largest finite float)
//   key_e = s_e + b_e, or x_e where nothing but the order of s_e matters (no bias, no sums of scores)
//   groups of E / G consecutive experts are ranked by their largest key or by the sum of their two
//   largest; the topk_groups best groups stay; the k largest keys in them are chosen, ties to the
//   lowest index
//   w_j   = scale * s_j / (renormalize ? sum over the chosen of s : 1)
//
// The choice is exact: it is what the definition gives in fp64. fp32 scores decide a token when every
// pair of keys whose order matters lies further apart than the fp32 error bound; otherwise (well under a
// percent of tokens, but one is enough to set a batch's time) the experts in doubt are ordered by fp64
// keys, or, where more than one left out or a group is in doubt, all of the choice is repeated in fp64.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "fastdiv.cuh"
#include "ptx.cuh"

namespace mx {

constexpr int kRouteThreads = 128;
constexpr int kRouteMaxTopk = 16;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxGroups = 32;
constexpr uint32_t kFullMask = 0xFFFFFFFFu;

struct RouteArgs {
    const void* x;            // logits [T, E], row stride ld
    const float* bias;        // [E] or null
    int32_t* ids;             // [T, k]
    float* w;                 // [T, k]
    int64_t T, ld;
    int E, k, G, topg;
    FastDiv per;              // experts per group
    int lanes_per_group;      // lanes whose experts make up one group (a power of two), 0: groups cut lanes
    int bf16, vec;            // element type; rows of NV experts per lane can be loaded as vectors
    int vec_bias;
    int sigmoid, top2, renorm;
    float scale;
    // backward
    const float* dw;          // [T, k]
    void* dx;                 // [T, E], row stride ld_dx
    int64_t ld_dx;
    int vec_dx;               // rows of four consecutive experts can be stored (vec: loaded) as vectors
};

// ---- rows of NV consecutive experts per lane ------------------------------------------------------

template <int BYTES>
struct RouteVec;
template <>
struct RouteVec<2> { using T = uint16_t; };
template <>
struct RouteVec<4> { using T = uint32_t; };
template <>
struct RouteVec<8> { using T = uint2; };
template <>
struct RouteVec<16> { using T = uint4; };

// Lane l's experts l * NV + i of row `base` (elements). Entries past E read -inf; NaN reads -inf and
// +inf the largest finite float, so that x - max and every sum stay defined.
template <int NV, class ELT>
__device__ __forceinline__ void route_load(const ELT* base, int E, int lane, bool vec, float (&v)[NV]) {
    constexpr int kBytes = NV * static_cast<int>(sizeof(ELT)) < 16 ? NV * static_cast<int>(sizeof(ELT)) : 16;
    constexpr int kPer = kBytes / static_cast<int>(sizeof(ELT));
    using V = typename RouteVec<kBytes>::T;
    const int e0 = lane * NV;
    ELT raw[NV];
    if (vec && e0 < E) {          // E is a multiple of NV here: a lane is all in or all out
#pragma unroll
        for (int c = 0; c < NV / kPer; ++c)
            *reinterpret_cast<V*>(&raw[c * kPer]) = reinterpret_cast<const V*>(base + e0)[c];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f = __int_as_float(0xFF800000);
        if (e0 + i < E) {
            const ELT r = vec ? raw[i] : base[e0 + i];
            f = sizeof(ELT) == 2 ? __uint_as_float(static_cast<uint32_t>(r) << 16) : __uint_as_float(static_cast<uint32_t>(r));
        }
        v[i] = f == f ? fminf(f, 3.402823466e38f) : __int_as_float(0xFF800000);
    }
}

__device__ __forceinline__ float route_logit(const RouteArgs& a, int64_t t, int e) {
    float f;
    if (a.bf16)
        f = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.x)[t * a.ld + e]) << 16);
    else
        f = static_cast<const float*>(a.x)[t * a.ld + e];
    return f == f ? fminf(f, 3.402823466e38f) : __int_as_float(0xFF800000);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// sigmoid(x) * e^-c for c <= 0, c >= x where x <= 0 (c = 0: the sigmoid). Dividing every score of a row by
// e^c, c = min(largest chosen logit, 0), keeps ratios of scores that themselves underflow.
__device__ __forceinline__ float route_sigmoid(float x, float c) {
    return x > 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - c) / (1.0f + expf(x));
}

// ---- ordered keys -------------------------------------------------------------------------------
// Unsigned integers in the order of the values (-0 equal to +0); 0 marks an expert that cannot be
// chosen (a key of -inf or NaN).

__device__ __forceinline__ uint32_t key_of(float f) {
    f += 0.0f;
    const uint32_t b = __float_as_uint(f);
    return f > __int_as_float(0xFF800000) ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ uint64_t key_of(double f) {
    f += 0.0;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(f));
    return f > __longlong_as_double(0xFFF0000000000000ll) ? ((b >> 63) ? ~b : b | 0x8000000000000000ull) : 0ull;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ double value_of(uint64_t k) {
    return __longlong_as_double(static_cast<long long>((k >> 63) ? k ^ 0x8000000000000000ull : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kFullMask, k); }
__device__ __forceinline__ uint32_t warp_min(uint32_t k) { return __reduce_min_sync(kFullMask, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kFullMask, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFullMask, (k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ __forceinline__ uint64_t warp_min(uint64_t k) { return ~warp_max(~k); }
template <class U>
__device__ __forceinline__ U shfl_xor(U v, int o) {
    return __shfl_xor_sync(kFullMask, v, o);
}

// Whether two keys lie too near together for fp32 to order them: also where the difference of two
// infinities or an overflowed sum says nothing.
__device__ __forceinline__ bool too_near(float hi, float lo, float tol) {
    return !(hi - lo > tol + 2.4e-7f * fmaxf(fabsf(hi), fabsf(lo)));
}

// Rank of a group whose two largest keys are m and c (0: there is no such expert).
template <class U>
__device__ __forceinline__ U group_rank(U m, U c, bool top2) {
    if (!top2 || c == 0) return m;
    const U s = key_of(value_of(m) + value_of(c));
    return s != 0 ? s : 1;           // a sum that overflows to -inf still ranks above a group without any expert
}

// Ranks the groups and clears the keys of all but the topg best. `last` and `next`: the ranks of the worst group
// kept and the best one left (0 if none). Where groups are whole lanes (a power of two of them), a group's two
// largest keys are merged over its lanes by shuffles; otherwise the keys go through a row of shared memory (8 bytes an
// expert and warp, for fp32 keys too: while one warp ranks fp64 keys its neighbours may still be at fp32 ones, and nothing
// orders warps) and lane g reads group g's. Every group then counts the groups before it with G independent
// shuffles. (Walking the groups with a warp maximum each took 4 us more for 5201 tokens of 10 groups of 10.)
extern __shared__ uint64_t route_smem[];

template <int NV, class U>
__device__ __forceinline__ void route_groups(const RouteArgs& a, U (&key)[NV], int lane, U& last, U& next) {
    const int G = a.G, L = a.lanes_per_group, per = static_cast<int>(a.per.d);
    const bool top2 = a.top2 != 0;
    U rank = 0;
    int mine = lane;                 // the group whose rank this lane holds
    if (L > 0) {
        U m = 0, c = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const U lo = key[i] < m ? key[i] : m;
            m = key[i] < m ? m : key[i];
            c = lo < c ? c : lo;
        }
        for (int o = 1; o < L; o <<= 1) {
            const U m2 = shfl_xor(m, o), c2 = shfl_xor(c, o);
            const U lo = m2 < m ? m2 : m, hi = m2 < m ? m : m2, cc = c2 < c ? c : c2;
            m = hi;
            c = lo < cc ? cc : lo;
        }
        rank = group_rank(m, c, top2);
        mine = lane / L;
    } else {
        U* row = reinterpret_cast<U*>(route_smem + (threadIdx.x >> 5) * a.E);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane * NV + i < a.E) row[lane * NV + i] = key[i];
        __syncwarp();
        if (lane < G) {
            U m = 0, c = 0;
            const U* mine_keys = row + lane * per;
#pragma unroll 4
            for (int j = 0; j < per; ++j) {
                const U k = mine_keys[j];
                const U lo = k < m ? k : m;
                m = k < m ? m : k;
                c = lo < c ? c : lo;
            }
            rank = group_rank(m, c, top2);
        }
        __syncwarp();
    }
    int before = 0;
    for (int g = 0; g < G; ++g) {
        const U r = __shfl_sync(kFullMask, rank, L > 0 ? g * L : g);
        before += r > rank || (r == rank && g < mine);
    }
    const bool kept = rank != 0 && before < a.topg;
    last = warp_min(kept ? rank : ~static_cast<U>(0));
    next = warp_max(kept ? static_cast<U>(0) : rank);
    const uint32_t mask = __ballot_sync(kFullMask, kept);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = L > 0 ? kept : ((mask >> (a.per.div(lane * NV + i) & 31u)) & 1u) != 0;
        if (!in) key[i] = 0;
    }
}

// The n largest keys, largest first, ties to the lowest index: lane j gets slot j's expert and key; they stay
// as they are where fewer experts can be chosen. Lanes hold consecutive experts, so the lowest lane that holds
// the maximum holds the lowest index, and inside a lane the tree keeps the lower one of equals. LEFT: also the best
// expert left out and its key (-1 and 0 if none), in every lane.
template <int NV, bool LEFT, class U>
__device__ __forceinline__ void route_select(U (&key)[NV], int n, int lane, int& id, U& slot_key, int& left, U& left_key) {
    left = -1;
    left_key = 0;
    for (int j = 0; j < n + (LEFT ? 1 : 0); ++j) {
        U b[NV];
        int bi[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            b[i] = key[i];
            bi[i] = i;
        }
#pragma unroll
        for (int h = 1; h < NV; h <<= 1)
#pragma unroll
            for (int i = 0; i < NV; i += 2 * h) {
                const bool right = b[i + h] > b[i];
                b[i] = right ? b[i + h] : b[i];
                bi[i] = right ? bi[i + h] : bi[i];
            }
        const U m = warp_max(b[0]);
        if (m == 0) break;
        const int owner = __ffs(__ballot_sync(kFullMask, b[0] == m)) - 1;
        const int e = __shfl_sync(kFullMask, lane * NV + bi[0], owner);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane * NV + i == e) key[i] = 0;
        if (LEFT && j == n) {
            left = e;
            left_key = m;
        } else if (lane == j) {
            id = e;
            slot_key = m;
        }
    }
}

// BF16 logits that decide by themselves: the key's 16 bits above the expert's index counted down, one word per
// expert, all different. One warp maximum then is the key, the expert and the tie rule at once. Each lane sorts
// its words (a network of 0, 1, 5 or 19 exchanges) and the winner's lane moves up its next.
// (key_of() + 0x8000) >> 16: BF16 values have 16 zero bits (ones below zero, which carry alike), and the largest
// finite float, which +inf stands for, rounds up past BF16's largest.
template <int NV>
__device__ __forceinline__ uint32_t packed_key(uint32_t key, int e) {
    return ((key + 0x8000u) & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(e));
}
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
template <int NV>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[NV]) {
    if constexpr (NV == 2) exchange(key[0], key[1]);
    if constexpr (NV == 4) {
        exchange(key[0], key[1]);
        exchange(key[2], key[3]);
        exchange(key[0], key[2]);
        exchange(key[1], key[3]);
        exchange(key[1], key[2]);
    }
    if constexpr (NV == 8) {
        constexpr int kNet[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                     {0, 4}, {3, 7}, {1, 5}, {2, 6}, {1, 4}, {3, 6}, {2, 4}, {3, 5}, {3, 4}};
#pragma unroll
        for (int i = 0; i < 19; ++i) exchange(key[kNet[i][0]], key[kNet[i][1]]);
    }
}
// The choice of TOK tokens at once (their chains of maxima run side by side): lane q * LPT + j gets token q's slot j
// as its packed key, 0 if there is none.
template <int NV, int TOK, int LPT>
__device__ __forceinline__ uint32_t route_select_packed(uint32_t (&key)[TOK][NV], int n, int lane) {
    constexpr bool kSorted = NV <= 8;
    if constexpr (kSorted) {
#pragma unroll
        for (int q = 0; q < TOK; ++q) sort_keys<NV>(key[q]);
    }
    uint32_t got = 0;
    for (int j = 0; j < n; ++j) {
        uint32_t m[TOK];
#pragma unroll
        for (int q = 0; q < TOK; ++q) {
            uint32_t b = key[q][0];
            if constexpr (!kSorted) {
#pragma unroll
                for (int i = 1; i < NV; ++i) b = max(b, key[q][i]);
            }
            m[q] = __reduce_max_sync(kFullMask, b);
        }
#pragma unroll
        for (int q = 0; q < TOK; ++q) {
            if (lane == q * LPT + j) got = m[q];
            if constexpr (kSorted) {
                if (key[q][0] == m[q]) {
#pragma unroll
                    for (int i = 0; i + 1 < NV; ++i) key[q][i] = key[q][i + 1];
                    key[q][NV - 1] = 0;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) key[q][i] = key[q][i] == m[q] ? 0u : key[q][i];
            }
        }
    }
    return got >= 0x10000u ? got : 0u;       // below: nothing was left that can be chosen
}

// fp64 arithmetic for tokens that fp32 cannot decide. One copy of each, not inlined: a few tokens of a batch come
// here, and what they cost is the time to fetch the instructions.
__device__ __noinline__ double route_exp(double x) { return exp(x); }
__device__ __noinline__ double route_quotient(double a, double b) { return a / b; }
// The row's softmax denominator (1 for a sigmoid) and the score of logit x.
template <int NV>
__device__ __forceinline__ double route_sum(const RouteArgs& a, const float (&v)[NV], float M) {
    if (a.sigmoid) return 1.0;
    double z = 0.0;
#pragma unroll 1
    for (int i = 0; i < NV; ++i)
        if (v[i] > __int_as_float(0xFF800000)) z += route_exp(static_cast<double>(v[i]) - static_cast<double>(M));
    return warp_sum(z);
}
__device__ __noinline__ double route_score(bool sigmoid, float x, float M, double z) {
    const double e = route_exp(sigmoid ? -static_cast<double>(x) : static_cast<double>(x) - static_cast<double>(M));
    return route_quotient(sigmoid ? 1.0 : e, sigmoid ? 1.0 + e : z);
}

// The choice in fp64, for a token that fp32 cannot decide: slot j's expert in lane j.
template <int NV>
__device__ __noinline__ int route_exact(const RouteArgs& a, const float (&v)[NV], float M, int lane) {
    const double kNone = __longlong_as_double(0xFFF0000000000000ll);
    const double z = route_sum(a, v, M);
    uint64_t key[NV];
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        double s = kNone;
        if (e < a.E && v[i] > __int_as_float(0xFF800000)) {
            s = route_score(a.sigmoid != 0, v[i], M, z);
            if (a.bias) s += static_cast<double>(a.bias[e]);
        }
        key[i] = key_of(s);
    }
    uint64_t last, next, slot_key = 0, left_key;
    if (a.G > 1) route_groups(a, key, lane, last, next);
    int id = -1, left;
    route_select<NV, false>(key, a.k, lane, id, slot_key, left, left_key);
    return id;
}

// The order of the k chosen experts (lanes 0 .. k - 1: id, logit x, bias b) and the best one left out (lane k) by
// fp64 keys: afterwards lane j < k holds the expert of slot j and its logit. All that is needed where no other
// expert's key comes near the last chosen one's. Lanes without an expert have id -1.
template <int NV>
__device__ __noinline__ void route_reorder(const RouteArgs& a, const float (&v)[NV], float M, int lane, int& id, float& x,
                                           float b) {
    const double z = route_sum(a, v, M);
    double key = __longlong_as_double(0xFFF0000000000000ll);
    if (id >= 0) {
        key = route_score(a.sigmoid != 0, x, M, z);
        if (a.bias) key += static_cast<double>(b);
    }
    int before = 0;
    for (int i = 0; i <= a.k; ++i) {
        const double o = __shfl_sync(kFullMask, key, i);
        const int oi = __shfl_sync(kFullMask, id, i);
        before += oi >= 0 && (o > key || (o == key && oi < id));
    }
    if (id < 0) before = 32 + lane;
    int from = lane;
    for (int i = 0; i <= a.k; ++i)
        if (__shfl_sync(kFullMask, before, i) == lane) from = i;
    id = __shfl_sync(kFullMask, id, from);
    x = __shfl_sync(kFullMask, x, from);
}

template <int NV>
__device__ __forceinline__ void route_load_row(const RouteArgs& a, int64_t t, int lane, float (&v)[NV]) {
    if (a.bf16)
        route_load<NV>(static_cast<const uint16_t*>(a.x) + t * a.ld, a.E, lane, a.vec != 0, v);
    else
        route_load<NV>(static_cast<const uint32_t*>(a.x) + t * a.ld, a.E, lane, a.vec != 0, v);
}

// A warp takes 32 / LPT tokens, LPT lanes for the slots of each. A row is spread over the whole warp, NV consecutive
// experts l * NV .. in lane l, while its experts are chosen; the slots' arithmetic and stores then run for all of
// the warp's tokens at once. PACKED: BF16 logits that decide by themselves.
//
// Bound by the choice's instructions and their latency, not by the one read of the logits (20 480 x 128 BF16 are
// 5 MB, less than a microsecond): some 25 instructions per chosen expert, 8 with packed keys, whose chains of maxima
// run side by side for the warp's tokens. Several tokens per warp are for large batches with packed keys and at most
// 128 experts: 20 480 x 128, top 8: 7.4 us with four tokens a warp, 9.5 us with one; 256 tokens: 3.4 and 2.1 us;
// 20 480 x 256: 15.4 and 15.1 us. Without packed keys a warp's tokens only queue up (sigmoid with bias, 20 480 x 128:
// 28.8 us with four where one took 23.1 us).
template <int NV, int LPT, bool PACKED>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const __grid_constant__ RouteArgs a) {
    grid_wait();
    constexpr int kTokens = 32 / LPT;
    static_assert(PACKED || kTokens == 1, "the general form takes one token per warp");
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5)) * kTokens;
    if (t0 >= a.T) return;
    const float kNone = __int_as_float(0xFF800000);
    const bool by_logit = a.bias == nullptr && !(a.G > 1 && a.top2);
    const bool row_softmax = !a.sigmoid && !(by_logit && a.renorm);     // the weights or keys need the row's sum
    int id = -1;
    float x = kNone, M = kNone, z = 0.0f;                               // the slot's expert and logit; its row's max, sum
    auto row_max_sum = [&](const float(&v)[NV], float(&f)[NV], float& m, float& sum) {
        // M of a row without any expert stays -inf and is never subtracted.
        m = kNone;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, v[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f[i] = v[i] > kNone ? expf(v[i] - m) : 0.0f;
            sum += f[i];
        }
        sum = warp_sum(sum);
    };
    if constexpr (PACKED) {
        uint32_t key[kTokens][NV];
#pragma unroll
        for (int q = 0; q < kTokens; ++q) {
            const int64_t t = t0 + q < a.T ? t0 + q : a.T - 1;
            float v[NV];
            route_load_row<NV>(a, t, lane, v);
            if (row_softmax) {
                float f[NV], m, sum;
                row_max_sum(v, f, m, sum);
                if (lane / LPT == q) {
                    M = m;
                    z = sum;
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) key[q][i] = packed_key<NV>(key_of(v[i]), lane * NV + i);
            if (a.G > 1) {
                // A group without any expert to choose must not be kept for its indices alone.
                uint32_t last, next;
#pragma unroll
                for (int i = 0; i < NV; ++i) key[q][i] = key[q][i] < 0x10000u ? 0u : key[q][i];
                route_groups(a, key[q], lane, last, next);
            }
        }
        const uint32_t got = route_select_packed<NV, kTokens, LPT>(key, a.k, lane);
        if (got != 0) {
            id = static_cast<int>(0xFFFFu - (got & 0xFFFFu));
            // The logit back from its key: positive as it was, negative less the rounding's carry, +inf's stand-in.
            const uint32_t top = got & 0xFFFF0000u;
            x = value_of(top >= 0xFF800000u ? 0xFF7FFFFFu : (top & 0x80000000u ? top : top - 1u));
        }
    } else {
        const int64_t t = t0;
        float v[NV], f[NV];
        route_load_row<NV>(a, t, lane, v);
        if (row_softmax) row_max_sum(v, f, M, z);
        uint32_t key[NV], last, next, slot_key = 0, left_key;
        int left;
        if (by_logit) {
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = key_of(v[i]);
            if (a.G > 1) route_groups(a, key, lane, last, next);
            route_select<NV, false>(key, a.k, lane, id, slot_key, left, left_key);
            if (slot_key != 0) x = value_of(slot_key);
        } else {
            float b[NV];
            if (a.bias) {
                route_load<NV>(reinterpret_cast<const uint32_t*>(a.bias), a.E, lane, a.vec_bias != 0, b);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) b[i] = 0.0f;
            }
            // |fp32 score - score|. Sigmoid, 1 / (1 + e^-x) with __expf (2 + 1.17 |x| ulp) and __fdividef (2 ulp):
            // s (1 - s) (2 + 1.17 |x|) 2^-23 <= 0.65 * 2^-23, + 2^-22 + 2^-24 < 3.9e-7. Softmax, of the row's largest
            // score 1 / z: expf and the sum's terms 2^-22 each, x - M rounded 2^-24 |x - M|, weighted by p in the score
            // (0.4) and in z (its mean is below ln 1024 = 6.9), the sum (NV + 5) 2^-24, two products 2^-23:
            // 1.4e-6 + 6e-8 NV. Twice that for a pair of keys, and twice again for a sum of two; the rounding of a
            // key, 2^-24 of it, is in too_near().
            float tol = a.sigmoid ? 8e-7f : (2.8e-6f + 1.2e-7f * NV) / z;
            if (a.G > 1 && a.top2) {
                // A sum of two keys also has its keys' roundings, which it may cancel below: 2^-24 of each and of
                // the sum, at most 4 * 2^-24 (1 + max |b|), twice that for a pair.
                float bm = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (v[i] > kNone && b[i] > kNone) bm = fmaxf(bm, fabsf(b[i]));
                bm = __uint_as_float(warp_max(__float_as_uint(bm)));
                tol = 2.0f * tol + 4.8e-7f * (1.0f + bm);
            }
            const float inv_z = 1.0f / z;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float s = a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-v[i])) : f[i] * inv_z;
                s = v[i] > kNone ? s + b[i] : kNone;
                key[i] = key_of(s);
            }
            bool near_group = false, near = false;
            if (a.G > 1) {
                route_groups(a, key, lane, last, next);
                near_group = next != 0 && too_near(value_of(last), value_of(next), tol);
            }
            route_select<NV, true>(key, a.k, lane, id, slot_key, left, left_key);
            // Lane k takes the best expert left out. Slot j against slot j + 1, the last one against lane k. Two
            // experts with the same logit and the same bias, twins, have the same score in any precision.
            if (lane == a.k) {
                id = left;
                slot_key = left_key;
            }
            float bj = 0.0f;
            if (id >= 0) {
                x = route_logit(a, t, id);
                if (a.bias) bj = a.bias[id];
            }
            const uint32_t k2 = __shfl_down_sync(kFullMask, slot_key, 1);
            const float x2 = __shfl_down_sync(kFullMask, x, 1), b2 = __shfl_down_sync(kFullMask, bj, 1);
            bool twins = false;              // the last chosen and the best left out are: others may stand right behind them
            if (lane < a.k && slot_key != 0 && k2 != 0) {
                if (x == x2 && bj == b2)
                    twins = lane == a.k - 1;
                else
                    near = too_near(value_of(slot_key), value_of(k2), tol);
            }
            if (__any_sync(kFullMask, near || twins || near_group)) {
                // Any other expert near the last chosen one (or a choice of groups in doubt): all of it in fp64. Where
                // nothing but twins at the border brought the token here, more twins of theirs (all logits equal, before
                // a router's first update) do not count: every one of them is behind the chosen by its index.
                const bool order = __any_sync(kFullMask, near);
                const float xb = __shfl_sync(kFullMask, x, a.k - 1), bb = __shfl_sync(kFullMask, bj, a.k - 1);
                uint32_t rest = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const bool twin = !order && key[i] != 0 && v[i] == xb && (!a.bias || a.bias[lane * NV + i] == bb);
                    rest = max(rest, twin ? 0u : key[i]);
                }
                rest = warp_max(left_key != 0 ? rest : 0u);
                const uint32_t border = __shfl_sync(kFullMask, slot_key, a.k - 1);
                if (near_group || (rest != 0 && left_key != 0 && too_near(value_of(border), value_of(rest), tol))) {
                    id = route_exact<NV>(a, v, M, lane);
                    x = id >= 0 ? route_logit(a, t, id) : kNone;
                } else if (order) {
                    route_reorder<NV>(a, v, M, lane, id, x, bj);
                }
            }
            if (lane >= a.k) x = kNone;
        }
    }
    const bool got = x > kNone;
    float s = 0.0f;
    if (a.renorm) {
        // Ratios of the chosen scores. Softmax: a softmax over the chosen alone.
        float m = x;
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
        if (got) s = a.sigmoid ? route_sigmoid(x, fminf(m, 0.0f)) : expf(x - m);
        float sum = s;
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        if (got) s /= sum;
    } else if (got) {
        s = a.sigmoid ? route_sigmoid(x, 0.0f) : expf(x - M) / z;
    }
    const int64_t t = t0 + lane / LPT;
    const int j = lane % LPT;
    if (t < a.T && j < a.k) {
        a.ids[t * a.k + j] = got ? id : -1;
        a.w[t * a.k + j] = a.scale * s;
    }
}

// Gradient of the weights with respect to the logits, the choice held fixed. With dw the incoming
// gradient and r_j = s_j / sum of the chosen s:
//   renormalized: c_j = scale * r_j * (dw_j - sum dw r); softmax: dx_j = c_j;
//                 sigmoid: dx_j = c_j * (1 - s_j); every other dx is 0;
//   otherwise:    sigmoid: dx_j = scale * dw_j * s_j (1 - s_j), others 0;
//                 softmax: dx_e = p_e * (d_e - sum_j d_j p_j) with d_j = scale * dw_j at the chosen.
// Only the last form reads whole rows; the others read the k chosen logits and write the row.
//
// A warp takes 32 / LPT tokens: LPT = 8 or 16 lanes, one per slot, for each, and the slots' arithmetic runs for all of
// them at once; LPT = 32, one token, in the last form, whose time is that of its row's exponentials (four tokens'
// rows in a warp took 8.5 us for 5201 x 100 and 6.3 us for 16 x 128, one 5.3 and 2.9; 20 480 x 128: 12.0 and 12.8).
// Then row by row: the chosen experts' parts are put into a row of zeros in shared memory, the row is
// read back four experts per lane, finished and stored, and the parts are cleared again. An expert named twice gets
// the sum of its parts in slot order.
template <int LPT>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_kernel(const __grid_constant__ RouteArgs a) {
    grid_wait();
    constexpr int kTokens = 32 / LPT;
    __shared__ __align__(16) float rows[kRouteThreads / 32][kRouteMaxExperts];
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5)) * kTokens;
    if (t0 >= a.T) return;
    const float kNone = __int_as_float(0xFF800000);
    float* buf = rows[threadIdx.x >> 5];
    const int q = lane / LPT, j = lane % LPT;
    int id = -1;
    float g = 0.0f, x = kNone;
    if (t0 + q < a.T && j < a.k) {
        const int64_t at = (t0 + q) * a.k + j;
        id = a.ids[at];
        g = a.dw[at];
        if (id >= 0 && id < a.E) x = route_logit(a, t0 + q, id);
    }
    const int chunks = (a.E + 127) / 128;                 // pieces of 128 experts, four per lane
    for (int c = 0; c < chunks; ++c) reinterpret_cast<float4*>(buf)[c * 32 + lane] = make_float4(0, 0, 0, 0);
    const bool got = x > kNone;
    if (!got) g = 0.0f;

    auto load4 = [&](int64_t t, int c, float(&v)[4]) {
        const int e0 = c * 128 + lane * 4;
        if (a.vec && e0 < a.E) {
            if (a.bf16) {
                const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + t * a.ld + e0);
                v[0] = __uint_as_float(r.x << 16);
                v[1] = __uint_as_float(r.x & 0xFFFF0000u);
                v[2] = __uint_as_float(r.y << 16);
                v[3] = __uint_as_float(r.y & 0xFFFF0000u);
            } else {
                const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + t * a.ld + e0);
                v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = v[i] == v[i] ? fminf(v[i], 3.402823466e38f) : kNone;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = e0 + i < a.E ? route_logit(a, t, e0 + i) : kNone;
        }
    };
    auto sum_slots = [&](float s) {
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
        return s;
    };
    constexpr bool kDense = LPT == 32;
    float c = 0.0f, row = 0.0f, M = kNone, z = 0.0f;      // the chosen expert's part; the row's sum of d p, max, sum
    if constexpr (kDense) {
        for (int ch = 0; ch < chunks; ++ch) {             // a running maximum and the sum relative to it
            float v[4];
            load4(t0, ch, v);
            const float mm = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), M);
            if (mm > M) z = M > kNone ? z * expf(M - mm) : 0.0f;
            M = mm;
#pragma unroll
            for (int i = 0; i < 4; ++i) z += v[i] > kNone ? expf(v[i] - mm) : 0.0f;
        }
        float mm = M;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(kFullMask, mm, o));
        z = warp_sum(M > kNone ? z * expf(M - mm) : 0.0f);
        M = mm;
        const float p = got ? expf(x - M) / z : 0.0f;
        c = a.scale * g * p;
        row = sum_slots(c);
    } else if (a.renorm) {
        float m = x;
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
        float s = 0.0f;
        if (got) s = a.sigmoid ? route_sigmoid(x, fminf(m, 0.0f)) : expf(x - m);
        const float sum = sum_slots(s);
        const float r = got ? s / sum : 0.0f;
        const float dot = sum_slots(g * r);
        c = a.scale * r * (g - dot);
        if (a.sigmoid && got) c *= route_sigmoid(-x, 0.0f);       // 1 - s
    } else if (got) {
        c = a.scale * g * route_sigmoid(x, 0.0f) * route_sigmoid(-x, 0.0f);
    }
    // An expert that two slots of a token name: the first one's lane gets the sum.
    const uint32_t same = __match_any_sync(kFullMask, got ? (static_cast<uint32_t>(q) << 16) | static_cast<uint32_t>(id)
                                                          : 0x80000000u | static_cast<uint32_t>(lane));
    bool put = got;
    if (__any_sync(kFullMask, __popc(same) > 1)) {
        put = got && lane == __ffs(same) - 1;
        float s = 0.0f;
        for (int jj = 0; jj < LPT; ++jj) {
            const float cj = __shfl_sync(kFullMask, c, q * LPT + jj);
            if ((same >> (q * LPT + jj)) & 1u) s += cj;
        }
        c = s;
    }
#pragma unroll
    for (int qq = 0; qq < kTokens; ++qq) {
        const int64_t t = t0 + qq;
        if (t >= a.T) break;
        if (put && q == qq) buf[id] = c;
        __syncwarp();
        for (int ch = 0; ch < chunks; ++ch) {
            const float4 o4 = reinterpret_cast<const float4*>(buf)[ch * 32 + lane];
            float o[4] = {o4.x, o4.y, o4.z, o4.w};
            if constexpr (kDense) {
                float v[4];
                load4(t, ch, v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (v[i] > kNone) o[i] -= expf(v[i] - M) / z * row;
            }
            const int e0 = ch * 128 + lane * 4;
            const int64_t at = t * a.ld_dx + e0;
            if (a.bf16) {
                uint16_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i]));
                uint16_t* dst = static_cast<uint16_t*>(a.dx) + at;
                if (a.vec_dx) {
                    if (e0 < a.E)
                        *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                                                                    h[2] | (static_cast<uint32_t>(h[3]) << 16));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e0 + i < a.E) dst[i] = h[i];
                }
            } else {
                float* dst = static_cast<float*>(a.dx) + at;
                if (a.vec_dx) {
                    if (e0 < a.E) *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e0 + i < a.E) dst[i] = o[i];
                }
            }
        }
        __syncwarp();
        if (put && q == qq) buf[id] = 0.0f;
        __syncwarp();
    }
}

// ---- the experts' row partition -------------------------------------------------------------------
//
// A stable counting sort of the n = T * k slots by expert: rows of expert e are its slots in slot
// order. Slots without an expert come after the last expert's rows and count as padding rows of the
// last group, so row_offsets always ends at n, as the grouped GEMMs require.
//   counts_kernel: every block counts the experts of its chunk of slots (n above one cluster's share);
//   plan_kernel:   every block adds up the counts of the blocks before it and of all blocks (the
//                  totals, whose scan are the offsets) and ranks the slots of its chunk. Up to 4096 slots
//                  take one block, up to 32 768 a cluster of 2, 4 or 8, which read one another's counts
//                  through distributed shared memory.
// Ranks come from per-warp counts in shared memory: a warp owns consecutive slots of the chunk and lanes
// with the same expert find one another by ballots, so the order never depends on timing.

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanOneBlock = 4096;       // slots that one block sorts by itself
constexpr int kPlanAhead = 4;             // loads of ids in flight per lane
constexpr int kPlanCluster = 8;           // blocks of the largest cluster that sorts without a counting kernel
constexpr int kPlanMaxBlocks = 128;

struct PlanArgs {
    const int32_t* ids;       // [n]
    int32_t* offsets;         // [E + 1]
    int32_t* slot_row;        // [n]
    int32_t* counts;          // [E]
    int32_t* block_counts;    // [blocks][E + 1] (workspace), null for one block
    int32_t n, E, chunk;
};

__device__ __forceinline__ int plan_bucket(const PlanArgs& a, int i) {
    const int id = a.ids[i];
    return id >= 0 && id < a.E ? id : a.E;
}

__global__ void __launch_bounds__(kPlanThreads) counts_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t plan_smem[];
    const int B = a.E + 1;
    grid_wait();
    for (int e = threadIdx.x; e < B; e += kPlanThreads) plan_smem[e] = 0;
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int hi = static_cast<int>(lo + a.chunk < a.n ? lo + a.chunk : a.n);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) atomicAdd(&plan_smem[plan_bucket(a, static_cast<int>(i))], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < B; e += kPlanThreads) a.block_counts[static_cast<int64_t>(blockIdx.x) * B + e] = plan_smem[e];
}

// Shared memory: warp counts [kPlanWarps][B], base [B], total [B], scan [kPlanWarps].
//
// Lanes with the same bucket are found by a ballot per bit of the bucket (match_any takes its time per distinct
// value: with 128 experts the one-block form spent 11.8 us on 4096 slots, most of it there).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t plan_smem[];
    const int B = a.E + 1;
    grid_wait();
    int32_t* wcount = plan_smem;
    int32_t* base = wcount + kPlanWarps * B;      // slots of the bucket in earlier blocks, then its first row here
    int32_t* total = base + B;
    int32_t* scan = total + B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < (kPlanWarps + 2) * B; i += kPlanThreads) plan_smem[i] = 0;
    __syncthreads();

    const int64_t blk_lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int64_t blk_hi = blk_lo + a.chunk < a.n ? blk_lo + a.chunk : a.n;
    const int per_warp = ((a.chunk + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int64_t lo = blk_lo + static_cast<int64_t>(warp) * per_warp;
    const int64_t hi = lo + per_warp < blk_hi ? lo + per_warp : blk_hi;
    // Buckets of this warp's next kPlanAhead x 32 slots (-1 past its end).
    auto load = [&](int64_t i0, int(&b)[kPlanAhead]) {
#pragma unroll
        for (int r = 0; r < kPlanAhead; ++r) {
            const int64_t i = i0 + 32 * r + lane;
            b[r] = i < hi ? plan_bucket(a, static_cast<int>(i)) : -1;
        }
    };
    const int bits = 32 - __clz(a.E);
    auto same_bucket = [&](int b) {
        uint32_t same = __ballot_sync(kFullMask, b >= 0);
        for (int i = 0; i < bits; ++i) {
            const bool one = (b >> i) & 1;
            const uint32_t ones = __ballot_sync(kFullMask, one);
            same &= one ? ones : ~ones;
        }
        return same;
    };
    int b[kPlanAhead];
    uint32_t same[kPlanAhead];
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kPlanAhead) {
        load(i0, b);
#pragma unroll
        for (int r = 0; r < kPlanAhead; ++r) same[r] = same_bucket(b[r]);
#pragma unroll
        for (int r = 0; r < kPlanAhead; ++r) {
            if (b[r] >= 0 && lane == __ffs(same[r]) - 1) wcount[warp * B + b[r]] += __popc(same[r]);
            __syncwarp();
        }
    }
    if (a.block_counts) {
        // Earlier blocks' and all blocks' counts of every bucket; a bucket's blocks are split over threads.
        const int blocks = gridDim.x, parts = kPlanThreads / B > 1 ? kPlanThreads / B : 1;
        for (int e = tid; e < B * parts; e += kPlanThreads) {
            const int b = e % B, part = e / B;
            int before = 0, all = 0;
#pragma unroll 8
            for (int j = part; j < blocks; j += parts) {
                const int c = a.block_counts[static_cast<int64_t>(j) * B + b];
                all += c;
                if (j < static_cast<int>(blockIdx.x)) before += c;
            }
            if (before) atomicAdd(&base[b], before);
            if (all) atomicAdd(&total[b], all);
        }
        __syncthreads();
    } else {
        __syncthreads();
        for (int e = tid; e < B; e += kPlanThreads) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kPlanWarps; ++w) sum += wcount[w * B + e];
            total[e] = sum;
        }
        __syncthreads();
        if (gridDim.x > 1) {
            // One cluster: this block's counts are its `total` until every block has read them.
            cluster_sync();
            int all[2] = {0, 0}, before[2] = {0, 0};         // B <= 1025: at most two buckets per thread
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = tid + i * kPlanThreads;
                if (e < B)
                    for (int r = 0; r < static_cast<int>(gridDim.x); ++r) {
                        const int c = static_cast<int>(ld_shared_cluster_u32(mapa_shared(smem_u32(&total[e]), r)));
                        all[i] += c;
                        if (r < static_cast<int>(blockIdx.x)) before[i] += c;
                    }
            }
            cluster_sync();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = tid + i * kPlanThreads;
                if (e < B) {
                    total[e] = all[i];
                    base[e] = before[i];
                }
            }
            __syncthreads();
        }
    }
    // Exclusive scan of the totals: first row of every bucket. B <= 1025: buckets past the first 1024
    // (only the last, "no expert") follow after the scan.
    const int mine = tid < B ? total[tid] : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int s = scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kFullMask, s, o);
            if (lane >= o) s += up;
        }
        scan[lane] = s;
    }
    __syncthreads();
    const int first = incl - mine + (warp > 0 ? scan[warp - 1] : 0);
    if (tid < B) base[tid] += first;
    if (tid == kPlanThreads - 1 && B > kPlanThreads) base[kPlanThreads] += first + mine;
    if (blockIdx.x == 0) {
        if (tid < a.E) {
            a.offsets[tid] = first;
            a.counts[tid] = mine;
        }
        if (tid == 0) a.offsets[a.E] = a.n;
    }
    __syncthreads();
    // First row of every (warp, bucket).
    for (int e = tid; e < B; e += kPlanThreads) {
        int row = base[e], c[kPlanWarps];
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) c[w] = wcount[w * B + e];
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            wcount[w * B + e] = row;
            row += c[w];
        }
    }
    __syncthreads();
    const bool once = per_warp <= 32 * kPlanAhead;       // buckets and lane masks are still in registers
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kPlanAhead) {
        if (!once) {
            load(i0, b);
#pragma unroll
            for (int r = 0; r < kPlanAhead; ++r) same[r] = same_bucket(b[r]);
        }
#pragma unroll
        for (int r = 0; r < kPlanAhead; ++r) {
            int row = 0;
            if (b[r] >= 0) row = wcount[warp * B + b[r]] + __popc(same[r] & ((1u << lane) - 1u));
            __syncwarp();
            if (b[r] >= 0 && lane == __ffs(same[r]) - 1) wcount[warp * B + b[r]] += __popc(same[r]);
            __syncwarp();
            if (b[r] >= 0) a.slot_row[i0 + 32 * r + lane] = b[r] < a.E ? row : ~row;
        }
    }
}

inline int plan_smem_bytes(int E) { return ((kPlanWarps + 2) * (E + 1) + kPlanWarps) * 4; }

}  // namespace mx
