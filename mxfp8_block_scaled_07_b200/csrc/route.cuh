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
// pair of keys whose order matters lies further apart than the fp32 error bound (kRouteTol below);
// otherwise (well under a percent of tokens) the warp repeats the choice with fp64 keys.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

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
    int bf16, vec;            // element type; rows of NV experts per lane can be loaded as vectors
    int sigmoid, top2, renorm;
    float scale;
    // backward
    const float* dw;          // [T, k]
    void* dx;                 // [T, E], row stride ld_dx
    int64_t ld_dx;
    int vec_dx;
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
            *reinterpret_cast<V*>(&raw[c * kPer]) = __ldg(reinterpret_cast<const V*>(base + e0) + c);
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
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kFullMask, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFullMask, (k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Whether two keys lie too near together for fp32 to order them: also where the difference of two
// infinities or an overflowed sum says nothing.
__device__ __forceinline__ bool too_near(float hi, float lo, float tol) {
    return !(hi - lo > tol + 2.4e-7f * fmaxf(fabsf(hi), fabsf(lo)));
}

// Ranks the groups and clears the keys of all but the topg best. `last` and `next`: the ranks of the
// worst group kept and the best one left (0 if none). Lane g ends up with group g's rank.
template <int NV, class U>
__device__ __forceinline__ void route_groups(U (&key)[NV], int G, int per, int topg, bool top2, int lane, U& last,
                                             U& next) {
    U rank = 0;
    for (int g = 0; g < G; ++g) {
        const int lo = g * per - lane * NV, hi = lo + per;      // the group's range in this lane's indices
        U b = 0;
        int bi = -1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i >= lo && i < hi && key[i] > b) {
                b = key[i];
                bi = i;
            }
        U m = warp_max(b);
        if (top2 && m != 0) {
            const int owner = __ffs(__ballot_sync(kFullMask, b == m)) - 1;
            U c = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i >= lo && i < hi && !(lane == owner && i == bi) && key[i] > c) c = key[i];
            c = warp_max(c);
            if (c != 0) {
                // A sum that overflows to -inf still ranks above a group without a choosable expert.
                const U s = key_of(value_of(m) + value_of(c));
                m = s != 0 ? s : 1;
            }
        }
        if (lane == g) rank = m;
    }
    uint32_t kept = 0;
    last = next = 0;
    for (int j = 0; j <= topg; ++j) {
        const U m = warp_max(rank);
        if (m == 0) break;
        if (j == topg) {
            next = m;
            break;
        }
        last = m;
        const int g = __ffs(__ballot_sync(kFullMask, rank == m)) - 1;
        kept |= 1u << g;
        if (lane == g) rank = 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = (lane * NV + i) / per;
        if (g >= 32 || !((kept >> g) & 1u)) key[i] = 0;
    }
}

// The n largest keys, largest first, ties to the lowest index: lane j < n gets slot j's expert and key
// (-1 and 0 when fewer experts can be chosen). Lanes hold consecutive experts, so the lowest lane that
// holds the maximum holds the lowest index.
template <int NV, class U>
__device__ __forceinline__ void route_select(U (&key)[NV], int n, int lane, int& id, U& slot_key) {
    id = -1;
    slot_key = 0;
    for (int j = 0; j < n; ++j) {
        U b = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (key[i] > b) {
                b = key[i];
                bi = i;
            }
        const U m = warp_max(b);
        if (m == 0) break;
        const int owner = __ffs(__ballot_sync(kFullMask, b == m)) - 1;
        const int e = __shfl_sync(kFullMask, lane * NV + bi, owner);
        if (lane == j) {
            id = e;
            slot_key = m;
        }
        if (lane == owner) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == bi) key[i] = 0;
        }
    }
}

// The choice in fp64, for a token that fp32 cannot decide.
template <int NV>
__device__ __noinline__ int route_exact(const RouteArgs& a, const float (&v)[NV], float M, int lane) {
    const double kNone = __longlong_as_double(0xFFF0000000000000ll);
    double z = 0.0;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int i = 0; i < NV; ++i)
            if (v[i] > __int_as_float(0xFF800000)) z += exp(static_cast<double>(v[i]) - static_cast<double>(M));
        z = warp_sum(z);
    }
    uint64_t key[NV];
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        double s = kNone;
        if (e < a.E && v[i] > __int_as_float(0xFF800000)) {
            const double x = static_cast<double>(v[i]);
            s = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(M)) / z;
            if (a.bias) s += static_cast<double>(a.bias[e]);
        }
        key[i] = key_of(s);
    }
    uint64_t last, next, slot_key;
    if (a.G > 1) route_groups(key, a.G, a.E / a.G, a.topg, a.top2 != 0, lane, last, next);
    int id;
    route_select(key, a.k, lane, id, slot_key);
    return id;
}

// One warp per token; lane l holds the NV consecutive experts l * NV .. of the row.
//
// Bound: one read of the logits. Measured figures and what they are made of stand with the entry point
// table of the design notes; at these sizes (a few MB) the selection's dependent warp reductions, two
// per chosen expert, weigh more than the bytes.
template <int NV>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const __grid_constant__ RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    float v[NV];
    if (a.bf16)
        route_load<NV>(static_cast<const uint16_t*>(a.x) + t * a.ld, a.E, lane, a.vec != 0, v);
    else
        route_load<NV>(static_cast<const uint32_t*>(a.x) + t * a.ld, a.E, lane, a.vec != 0, v);

    const float kNone = __int_as_float(0xFF800000);
    const bool by_logit = a.bias == nullptr && !(a.G > 1 && a.top2);
    float M = kNone, z = 0.0f;
    if (!a.sigmoid && !(by_logit && a.renorm)) {
        // Softmax over the row. M of a row without any expert stays -inf and is never subtracted.
#pragma unroll
        for (int i = 0; i < NV; ++i) M = fmaxf(M, v[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
#pragma unroll
        for (int i = 0; i < NV; ++i) z += v[i] > kNone ? expf(v[i] - M) : 0.0f;
        z = warp_sum(z);
    }
    uint32_t key[NV];
    float tol = 0.0f;
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = key_of(v[i]);
    } else {
        // |fp32 score - score|: sigmoid below 2.5e-7 (x > 0: half of expf's 2 ulp, 2^-23, and two roundings,
        // 2^-23, of a score of at most 1; x <= 0: 2^-22 and 2^-23 of at most a half); softmax at
        // most (2^-22 expf + 5 * 2^-24 from rounded x - max weighted by p + (NV + 5) * 2^-24 from the
        // sum + 2^-24 from the division) of the row's largest score 1 / z. Twice that for a pair; the
        // rounding of the sum with the bias, 2^-24 of each key, is in too_near(); twice all for a sum of two.
        tol = a.sigmoid ? 5e-7f : (1.4e-6f + 1.2e-7f * NV) / z;
        if (a.G > 1 && a.top2) tol *= 2.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane * NV + i;
            float s = kNone;
            if (e < a.E && v[i] > kNone) {
                s = a.sigmoid ? route_sigmoid(v[i], 0.0f) : expf(v[i] - M) / z;
                if (a.bias) s += a.bias[e];
            }
            key[i] = key_of(s);
        }
    }
    bool near = false;
    if (a.G > 1) {
        uint32_t last, next;
        route_groups(key, a.G, a.E / a.G, a.topg, a.top2 != 0, lane, last, next);
        if (!by_logit && next != 0) near = too_near(value_of(last), value_of(next), tol);
    }
    int id;
    uint32_t slot_key;
    route_select(key, by_logit ? a.k : a.k + 1, lane, id, slot_key);
    float x = kNone;
    if (id >= 0) x = route_logit(a, t, id);
    if (!by_logit) {
        // Slot j against slot j + 1; slot k is the best expert left out. Two experts with the same logit
        // and the same bias have the same score in any precision.
        const float b = id >= 0 && a.bias ? a.bias[id] : 0.0f;
        const uint32_t k2 = __shfl_down_sync(kFullMask, slot_key, 1);
        const float x2 = __shfl_down_sync(kFullMask, x, 1), b2 = __shfl_down_sync(kFullMask, b, 1);
        if (lane < a.k && slot_key != 0 && k2 != 0 && !(x == x2 && b == b2))
            near |= too_near(value_of(slot_key), value_of(k2), tol);
        if (__any_sync(kFullMask, near)) {
            id = route_exact<NV>(a, v, M, lane);
            x = id >= 0 && lane < a.k ? route_logit(a, t, id) : kNone;
        }
    }
    if (lane >= a.k) x = kNone;
    const bool got = x > kNone;
    float s = 0.0f;
    if (a.renorm) {
        // Ratios of the chosen scores. Softmax: a softmax over the chosen alone.
        float m = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
        if (got) s = a.sigmoid ? route_sigmoid(x, fminf(m, 0.0f)) : expf(x - m);
        const float sum = warp_sum(s);
        if (got) s /= sum;
    } else if (got) {
        s = a.sigmoid ? route_sigmoid(x, 0.0f) : expf(x - M) / z;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = got ? id : -1;
        a.w[t * a.k + lane] = a.scale * s;
    }
}

// Gradient of the weights with respect to the logits, the choice held fixed. With dw the incoming
// gradient and r_j = s_j / sum of the chosen s:
//   renormalized: ds-part c_j = scale * r_j * (dw_j - sum dw r); softmax: dx_j = c_j;
//                 sigmoid: dx_j = c_j * (1 - s_j); every other dx is 0;
//   otherwise:    sigmoid: dx_j = scale * dw_j * s_j (1 - s_j), others 0;
//                 softmax: dx_e = p_e * (d_e - sum_j d_j p_j) with d_j = scale * dw_j at the chosen.
// Only the last form reads the whole row; the others read the k chosen logits and write the row.
template <int NV>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_kernel(const __grid_constant__ RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const float kNone = __int_as_float(0xFF800000);
    int id = -1;
    float g = 0.0f, x = kNone;
    if (lane < a.k) {
        id = a.ids[t * a.k + lane];
        if (id < 0 || id >= a.E) id = -1;
        if (id >= 0) {
            x = route_logit(a, t, id);
            if (x > kNone) g = a.dw[t * a.k + lane];
        }
    }
    const bool got = x > kNone;
    float out[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) out[i] = 0.0f;
    float c = 0.0f, row = 0.0f;              // chosen expert's own part; what every expert's p is multiplied with
    float v[NV], M = kNone, z = 1.0f;
    const bool dense = !a.sigmoid && !a.renorm;
    if (dense) {
        if (a.bf16)
            route_load<NV>(static_cast<const uint16_t*>(a.x) + t * a.ld, a.E, lane, a.vec != 0, v);
        else
            route_load<NV>(static_cast<const uint32_t*>(a.x) + t * a.ld, a.E, lane, a.vec != 0, v);
#pragma unroll
        for (int i = 0; i < NV; ++i) M = fmaxf(M, v[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = v[i] > kNone ? expf(v[i] - M) : 0.0f;
            z += v[i];
        }
        z = warp_sum(z);
        const float p = got ? expf(x - M) / z : 0.0f;
        c = a.scale * g * p;
        row = warp_sum(c);
    } else if (a.renorm) {
        float m = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
        float s = 0.0f;
        if (got) s = a.sigmoid ? route_sigmoid(x, fminf(m, 0.0f)) : expf(x - m);
        const float sum = warp_sum(s);
        const float r = got ? s / sum : 0.0f;
        const float dot = warp_sum(g * r);
        c = a.scale * r * (g - dot);
        if (a.sigmoid && got) c *= route_sigmoid(-x, 0.0f);       // 1 - s
    } else if (got) {
        c = a.scale * g * route_sigmoid(x, 0.0f) * route_sigmoid(-x, 0.0f);
    }
    for (int j = 0; j < a.k; ++j) {
        const int e = __shfl_sync(kFullMask, id, j) - lane * NV;
        const float cj = __shfl_sync(kFullMask, c, j);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i == e) out[i] += cj;
    }
    if (dense && z > 0.0f) {
#pragma unroll
        for (int i = 0; i < NV; ++i) out[i] -= v[i] / z * row;
    }
    const int e0 = lane * NV;
    if (a.bf16) {
        uint16_t h[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(out[i]));
        uint16_t* dst = static_cast<uint16_t*>(a.dx) + t * a.ld_dx + e0;
        constexpr int kBytes = NV * 2 < 16 ? NV * 2 : 16;
        using V = typename RouteVec<kBytes>::T;
        if (a.vec_dx) {
            if (e0 < a.E)
#pragma unroll
                for (int q = 0; q < NV * 2 / kBytes; ++q)
                    reinterpret_cast<V*>(dst)[q] = *reinterpret_cast<const V*>(&h[q * (kBytes / 2)]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e0 + i < a.E) dst[i] = h[i];
        }
    } else {
        float* dst = static_cast<float*>(a.dx) + t * a.ld_dx + e0;
        constexpr int kBytes = NV * 4 < 16 ? NV * 4 : 16;
        using V = typename RouteVec<kBytes>::T;
        if (a.vec_dx) {
            if (e0 < a.E)
#pragma unroll
                for (int q = 0; q < NV * 4 / kBytes; ++q)
                    reinterpret_cast<V*>(dst)[q] = *reinterpret_cast<const V*>(&out[q * (kBytes / 4)]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e0 + i < a.E) dst[i] = out[i];
        }
    }
}

// ---- the experts' row partition -------------------------------------------------------------------
//
// A stable counting sort of the n = T * k slots by expert: rows of expert e are its slots in slot
// order. Slots without an expert come after the last expert's rows and count as padding rows of the
// last group, so row_offsets always ends at n, as the grouped GEMMs require.
//   counts_kernel: every block counts the experts of its chunk of slots (n above one block's share);
//   plan_kernel:   every block adds up the counts of the blocks before it and of all blocks (the
//                  totals, whose scan are the offsets) and ranks the slots of its chunk.
// Ranks come from per-warp counts in shared memory: a warp owns consecutive slots of the chunk, lanes
// with the same expert find one another with match_any, so the order never depends on timing.

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanOneBlock = 4096;       // slots that one block sorts by itself
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
    for (int e = threadIdx.x; e < B; e += kPlanThreads) plan_smem[e] = 0;
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int hi = static_cast<int>(lo + a.chunk < a.n ? lo + a.chunk : a.n);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) atomicAdd(&plan_smem[plan_bucket(a, static_cast<int>(i))], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < B; e += kPlanThreads) a.block_counts[static_cast<int64_t>(blockIdx.x) * B + e] = plan_smem[e];
}

// Shared memory: warp counts [kPlanWarps][B], base [B], total [B], scan [kPlanWarps].
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t plan_smem[];
    const int B = a.E + 1;
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
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const bool ok = i0 + lane < hi;
        const int b = ok ? plan_bucket(a, static_cast<int>(i0 + lane)) : -1;
        const uint32_t same = __match_any_sync(kFullMask, b);
        if (ok && lane == __ffs(same) - 1) wcount[warp * B + b] += __popc(same);
        __syncwarp();
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
            for (int w = 0; w < kPlanWarps; ++w) sum += wcount[w * B + e];
            total[e] = sum;
        }
        __syncthreads();
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
        int row = base[e];
        for (int w = 0; w < kPlanWarps; ++w) {
            const int c = wcount[w * B + e];
            wcount[w * B + e] = row;
            row += c;
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const bool ok = i0 + lane < hi;
        const int b = ok ? plan_bucket(a, static_cast<int>(i0 + lane)) : -1;
        const uint32_t same = __match_any_sync(kFullMask, b);
        int row = 0;
        if (ok) row = wcount[warp * B + b] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (ok && lane == __ffs(same) - 1) wcount[warp * B + b] += __popc(same);
        __syncwarp();
        if (ok) a.slot_row[i0 + lane] = b < a.E ? row : ~row;
    }
}

inline int plan_smem_bytes(int E) { return ((kPlanWarps + 2) * (E + 1) + kPlanWarps) * 4; }

}  // namespace mx
