// Attention over the paged E4M3 cache for many rows per sequence: prompts, and pieces of them.
//
// The mathematics is attend.cuh's; here the products decide: 4 D flops per row and key, on tcgen05. The unit of work is 256 query
// rows of one sequence and key head (256 / G tokens), two tiles of 128, whose keys are walked in tiles of 128:
//   S_t = Q_t K^T        tcgen05.mma kind::f16, both operands in shared memory, accumulators in TMEM
//   P_t = 2^(S_t ...)    one thread per row, read from TMEM and written back over S_t as f16
//   O_t += P_t V         P_t from TMEM, V from shared memory as it lies (features contiguous: an MN-major operand)
// While the softmax of one tile runs, the products of the other do. One warp copies the codes with bulk copies of 16 keys each,
// so that pages may be of any size from 16 tokens and lie anywhere; four warps write them to the products' layout as f16 (exact, one
// conversion for two codes). The scales stay out of the products: a page's key scale is a factor of the softmax's argument, its
// value scale's exponent part of P's, both constant over 16 columns. E4M3 operands would run at twice the rate but P (and q) would need two of
// them each to keep BF16's accuracy, which costs the softmax's threads more than the conversion costs the converters.
//
// Roles (512 threads): warps 0-3 and 4-7 softmax of tiles 0 and 1, warps 8-11 conversion, warp 12 issues the products and owns TMEM
// (S_0, S_1: 128 columns each, O_0, O_1: D each), warp 13 copies, warps
// 14 and 15 complete their warpgroup. The launch's 128 registers a thread are split 168 / 88 / 88 (8 x 168 + 4 x 88 + 4 x 88 = 16 x
// 128), without which the softmax spills. Every wait is bounded.
//
// 2048 rows x 32 heads of 128 against 16 000 keys (504 GFLOP): 562 us, 897 TFLOP/s, 0.55 of the dense rate in bursts. Of the 4600 cycles
// that a tile takes the products of both halves need 2048 and each half's softmax 3100; the rest a half waits for its next scores, which are
// made only once its second weights have been multiplied (P lies over the scores' columns) and behind the other half's products.
#pragma once
#include <cstdint>
#include <type_traits>

#include "attend.cuh"
#include "ptx.cuh"

namespace mx {

constexpr int kAmThreads = 512;
constexpr int kAmRing = 2;             // stages of K and of V
constexpr int kAmRaw = 4;              // half tiles of codes on their way to the loaders
constexpr int kAmScales = 4;           // tiles whose page scales are kept
constexpr uint32_t kAmCols = 512;
constexpr int kAmMinCost = 8;          // that a block takes at least
constexpr float kAmMost = 32768.0f;     // sum of 16 weights that sends M up: no weight passes f16's range
constexpr float kAmMostSum = 1.1e12f;   // 2^kAtSumSlack: what 64 keys add to l, beyond which its reference goes up
constexpr int kAmScaleRow = 10;         // of a tile: 8 groups' (key factor, value exponent), then a bit per group whose values are NaN

template <int D>
struct AmSmem {
    static constexpr int kTile = 128 * D * 2;                      // 128 rows of f16
    static constexpr int kQ = 0;                                   // two tiles
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kAmRing * kTile;
    static constexpr int kRaw = kV + kAmRing * kTile;              // codes of half tiles on their way
    static constexpr int kHalf = 64 * D;
    static constexpr int kScales = kRaw + kAmRaw * kHalf;          // [kAmScales][kAmScaleRow]
    static constexpr int kBar = kScales + kAmScales * kAmScaleRow * 8;
    static constexpr int kBars = 2 * kAmRaw + 4 * kAmRing + kAmScales + 14 + 1;
    static constexpr int kMisc = kBar + kBars * 8;
    static constexpr int kBytes = kMisc + 8 + 4 * kAmScales + 1024;    // + alignment slack
};

// ---- f16 products --------------------------------------------------------------------------------------------

__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool b_mn_major) {
    return (1u << 4)                              // accumulators: fp32; both operands f16 (format code 0)
           | (b_mn_major ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// MN-major operand in the 128-byte swizzle: rows (along K) of 128 bytes, 8-row groups 1024 bytes apart, the next 64 elements
// of MN one tile of 128 rows (16 KB) further.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(16384u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// D / 16 products S (+)= Q K^T of 16 features each and the commit on `bar`, under one election: adesc and bdesc are those of
// the first 16 features; the next lie 32 bytes on, the 64 behind them one tile half (16 KB) on.
template <int D>
__device__ __forceinline__ void tc_scores_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint64_t* bar) {
    if constexpr (D == 128)
        asm volatile(
            "{\n\t.reg .pred e, t, f;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\tadd.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, 1024;\n\tadd.s64 b5, %2, 1026;\n\tadd.s64 b6, %2, 1028;\n\tadd.s64 b7, %2, 1030;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, t;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(smem_u32(bar))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, t, f;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(smem_u32(bar))
            : "memory");
}
// Four products O (+)= P V of 16 keys each: P's next 16 keys lie 8 columns on, V's 2 KB on.
__device__ __forceinline__ void tc_values_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, t, p;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Pairs of fp32 in a 64-bit register: a b + c, and a + b. (Packed by themselves and not within the arithmetic's asm, which moved
// every operand anew each time.)
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Bits of 32 columns from `at` on that lie in [begin, end).
__device__ __forceinline__ uint32_t seen_bits(int begin, int end, int at) {
    const int lo = min(max(begin - at, 0), 32), hi = min(max(end - at, 0), 32);
    return hi <= lo ? 0u : (0xFFFFFFFFu >> (32 - (hi - lo))) << lo;
}

// ---- the block's work ------------------------------------------------------------------------------------------

// a / b for quotients below 1024 (key heads): a 64-bit division is 70 instructions, and every role divides.
__device__ __forceinline__ int quotient(int64_t a, int64_t b) {
    int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    while (q * b > a) --q;
    while ((q + 1) * b <= a) ++q;
    return q;
}

// A block walks its share [x, end) of all units' cost: a piece of a unit first, whole units, a piece last. Each role walks by
// itself. A share that ends within the cost in front of a unit's tiles leaves them all to the next block.
struct AmWork : AmItem {
    int h, N;                            // key head; tiles of this piece
    int64_t from;                        // first key of the piece
    int part[2];                         // tiles of either half of the rows within the piece
    bool begins, whole;                  // the piece is the unit's beginning, all of it
};
struct AmWalk {
    int64_t x, end;
    int item;
};
__device__ __forceinline__ bool next_piece(const AttendArgs& a, AmWalk& at, AmWork& w) {
    while (at.x < at.end) {
        static_cast<AmItem&>(w) = *plan_item(a, at.item);
        const int64_t cost = unit_cost(w);
        if (at.x >= w.at + cost * a.c.Hkv) {
            ++at.item;                   // there is one: x lies below the total
            continue;
        }
        w.h = quotient(at.x - w.at, cost);
        const int64_t s0 = w.at + w.h * cost, p1 = min(cost, at.end - s0);
        const int j0 = static_cast<int>(max(at.x - s0 - kAmUnitCost, int64_t(0))), j1 = static_cast<int>(max(p1 - kAmUnitCost, int64_t(0)));
        at.x = s0 + p1;
        if (j1 <= j0) continue;
        w.N = j1 - j0;
        w.from = w.lo + int64_t(j0) * kAmKeys;
#pragma unroll
        for (int t = 0; t < 2; ++t) w.part[t] = min(max(w.tiles[t] - j0, 0), w.N);
        w.begins = j0 == 0;
        w.whole = w.N == unit_tiles(w);
        return true;
    }
    return false;
}
__device__ __forceinline__ int64_t many_share(const AttendArgs& a, int64_t total) {
    return max((total + a.many_blocks - 1) / a.many_blocks, int64_t(kAmMinCost));
}
// The item that holds place x of the cost, by a whole block.
__device__ __forceinline__ int find_item(const AttendArgs& a, int items, int64_t x) {
    int n = 0;
    for (int i = 0; i < items; i += blockDim.x) {
        const int k = i + static_cast<int>(threadIdx.x);
        n += __syncthreads_count(k < items && plan_item(a, k)->at <= x);
    }
    return n - 1;
}
// Floats of a part: O [D / 4][256 rows][4], then M, l and lift of the rows.
__host__ __device__ constexpr int64_t many_part_floats(int D) { return int64_t(kAmRows) * (D + 3); }

// Order in which tiles of keys and values are copied and converted: K 0, then K j + 1 and V j for j = 0, 1, ..., without K N.
__device__ __forceinline__ int tile_of(int item, int N, bool& keys) {
    keys = item == 0 || (item % 2 == 1 && item < 2 * N - 1);
    return item == 0 ? 0 : item == 2 * N - 1 ? N - 1 : keys ? (item + 1) / 2 : item / 2 - 1;
}
// A bulk copy of one lane's.
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* gsrc, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kAmThreads, 1) attend_many_kernel(const __grid_constant__ AttendArgs a) {
    grid_wait();
    using S = AmSmem<D>;
    extern __shared__ uint8_t dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + S::kBar);
    uint64_t* raw_empty = raw_full + kAmRaw;
    uint64_t* k_full = raw_empty + kAmRaw;
    uint64_t* k_empty = k_full + kAmRing;
    uint64_t* v_full = k_empty + kAmRing;
    uint64_t* v_empty = v_full + kAmRing;
    uint64_t* scales_full = v_empty + kAmRing;
    uint64_t* q_full = scales_full + kAmScales;
    uint64_t* s_full = q_full + 2;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 4;               // p_full, o_done: of two halves of either tile
    uint64_t* q_seen = o_done + 4;               // the products' issuer has seen q_full
    uint64_t* drain = q_seen + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
    uint32_t* bad_pages = reinterpret_cast<uint32_t*>(smem + S::kMisc + 8);      // of a tile: a bit per group of 16 keys
    float2* scales = reinterpret_cast<float2*>(smem + S::kScales);
    const CacheView& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    AmWalk mine;
    {
        const int64_t total = plan_header(a)->total, share = many_share(a, total);
        mine.x = blockIdx.x * share;
        mine.end = min(mine.x + share, total);
        if (mine.x >= mine.end) return;
        mine.item = find_item(a, plan_header(a)->items, mine.x);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kAmRaw; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int i = 0; i < kAmRing; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kAmScales; ++i) mbar_init(&scales_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&q_seen[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_done[2 * i], 1);
            mbar_init(&o_done[2 * i + 1], 1);
        }
        mbar_init(drain, 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == 12) {
        tmem_alloc(tmem_slot, kAmCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        // ---- convert: codes of half tiles, as they lie in their pages, to f16 in the products' layout
        constexpr int U = 64 * D / 16 / 128;                 // 16-byte pieces per thread and half tile
        constexpr int R = 2048 / D;                          // rows that the four warps take at once: 16 or 32
        // Eight lanes: two rows and four pieces, so that their f16 meets every bank once under the swizzle.
        const int row_in = (warp - 8) * (R / 4) + (D == 128 ? ((lane >> 2) & 1) + 2 * (lane >> 4) : lane >> 2);
        const int piece = D == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : lane & 3;
        const uint32_t from = smem_u32(smem) + S::kRaw + row_in * D + piece * 16;
        const uint32_t to = (piece >> 2) * 16384 + row_in * 128;
        const uint32_t to0 = to + ((((piece & 3) * 2) ^ (row_in & 7)) << 4), to1 = to + ((((piece & 3) * 2 + 1) ^ (row_in & 7)) << 4);
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        int base = 0;                                        // tiles of the pieces in front
        AmWork w{};
        while (ok && next_piece(a, mine, w)) {
#pragma unroll 1
          for (int item = 0; ok && item < 2 * w.N; ++item) {
            bool keys;
            const int in = tile_of(item, w.N, keys), j = base + in, st = j % kAmRing;
            if (j >= kAmRing) ok = mbar_wait_warp(keys ? &k_empty[st] : &v_empty[st], (j / kAmRing - 1) & 1, abort, a.err, a.timeout_ns);
            if (!ok) break;
            const uint32_t tile = smem_u32(smem) + (keys ? S::kK : S::kV) + st * S::kTile;
            const int64_t left = w.hi - (w.from + int64_t(in) * kAmKeys);       // keys from the tile's first on
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                ok = mbar_wait_warp(&raw_full[stage], phase, abort, a.err, a.timeout_ns);
                if (!ok) break;
                uint4 x[U];
#pragma unroll
                for (int i = 0; i < U; ++i) x[i] = ld_shared_v4(from + stage * S::kHalf + i * 2048);
                // Behind the sequence's end nothing was copied, nor from a bad page (whose scales say NaN): zeros.
                if (left < kAmKeys || bad_pages[j % kAmScales] != 0) {
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int row = half * 64 + i * R + row_in;
                        if (row >= left || (bad_pages[j % kAmScales] >> (row >> 4) & 1)) x[i] = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const uint32_t at = tile + half * 8192 + i * R * 128;
                    st_shared_v4(at + to0, f16x2_of_e4m3(x[i].x), f16x2_of_e4m3_hi(x[i].x), f16x2_of_e4m3(x[i].y), f16x2_of_e4m3_hi(x[i].y));
                    st_shared_v4(at + to1, f16x2_of_e4m3(x[i].z), f16x2_of_e4m3_hi(x[i].z), f16x2_of_e4m3(x[i].w), f16x2_of_e4m3_hi(x[i].w));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&raw_empty[stage]);
                if (++stage == kAmRaw) stage = 0, phase ^= 1;
            }
            if (!ok) break;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(keys ? &k_full[st] : &v_full[st]);
          }
          base += w.N;
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 12) {
        // ---- products
        constexpr uint32_t idesc_s = idesc_f16(128, kAmKeys, false), idesc_o = idesc_f16(128, D, true);
        const uint32_t sm = smem_u32(smem);
        const uint64_t q_desc = sdesc_kmajor_sw128(sm + S::kQ), k_desc = sdesc_kmajor_sw128(sm + S::kK), v_desc = sdesc_mnmajor_sw128(sm + S::kV);
        auto scores = [&](int t, int st) {
            tc_scores_elect<D>(tmem + t * 128, q_desc + t * (S::kTile >> 4), k_desc + st * (S::kTile >> 4), idesc_s, &s_full[t]);
        };
        bool ok = true;
        int base = 0, turn = 0, seen[2] = {0, 0};            // tiles and pieces in front; tiles of either half of the rows
        AmWork w{};
        while (ok && next_piece(a, mine, w)) {
            ok = mbar_wait_warp(&q_full[0], turn & 1, abort, a.err, a.timeout_ns) && mbar_wait_warp(&q_full[1], turn & 1, abort, a.err, a.timeout_ns) &&
                 mbar_wait_warp(&k_full[base % kAmRing], (base / kAmRing) & 1, abort, a.err, a.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                mbar_arrive(&q_seen[0]);
                mbar_arrive(&q_seen[1]);
            }
            __syncwarp();
#pragma unroll 1
            for (int t = 0; t < 2; ++t)
                if (w.part[t] > 0) scores(t, base % kAmRing);
            tc_commit_elect(&k_empty[base % kAmRing]);
#pragma unroll 1
            for (int in = 0; ok && in < w.N; ++in) {
                const int j = base + in, vs = j % kAmRing, kn = (j + 1) % kAmRing;
                ok = mbar_wait_warp(&v_full[vs], (j / kAmRing) & 1, abort, a.err, a.timeout_ns);
                if (!ok) break;
                bool have_k = false;
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    if (in < w.part[t]) {
                        const uint64_t v_tile = v_desc + vs * (S::kTile >> 4);
#pragma unroll 1
                        for (int half = 0; ok && half < 2; ++half) {
                            ok = mbar_wait_warp(&p_full[2 * t + half], (seen[t] + in) & 1, abort, a.err, a.timeout_ns);
                            if (!ok) break;
                            tc_fence_after();
                            tc_values_elect(tmem + 256 + t * D, tmem + t * 128 + 32 * half, v_tile + 512 * half, idesc_o, in != 0 || half != 0);
                            tc_commit_elect(&o_done[2 * t + half]);
                        }
                        if (!ok) break;
                    }
                    if (in + 1 < w.part[t]) {
                        if (!have_k) {
                            ok = mbar_wait_warp(&k_full[kn], ((j + 1) / kAmRing) & 1, abort, a.err, a.timeout_ns);
                            if (!ok) break;
                            have_k = true;
                            tc_fence_after();
                        }
                        scores(t, kn);
                    }
                }
                if (!ok) break;
                tc_commit_elect(&v_empty[vs]);
                if (have_k) tc_commit_elect(&k_empty[kn]);
            }
            base += w.N;
            ++turn;
            seen[0] += w.part[0];
            seen[1] += w.part[1];
        }
        // Every product issued by this warp has completed once `drain` fires.
        tc_commit_elect(drain);
        mbar_wait_drain(drain, 0, a.timeout_ns);
        __syncwarp();
        } else if (warp == 13) {
        // ---- copy: lane l < 8 copies the 16 keys of group l, half a tile (four lanes) at a time, and brings the page scales
        AmWork w{};
        int id_next = -1;                                    // page of group `lane`, of the tile behind the last one placed
        uint32_t ks_next = 255, vs_next = 255, ks = 255, vs = 255;       // scale bytes of the tile last placed and of the one in front of it
        struct Place {
            int64_t k, v;                                    // of the lane's group: bytes from the codes' beginning
            int bytes;                                       // to copy: 0 outside the sequence or on a bad page
            uint32_t bad;
        };
        // Neither an id nor the scales are looked at where they are loaded: a tile later they have come.
        auto fetch_id = [&](int j) {
            const int64_t tok = w.from + int64_t(j) * kAmKeys + 16 * lane, index = tok >> c.page_shift;
            id_next = -1;
            if (lane < 8 && j < w.N && tok < w.hi && index < c.width) id_next = c.table[w.b * c.ld_table + index];
        };
        auto place = [&](int j) {                            // from id_next; then fetches the next tile's
            const int64_t tok = w.from + int64_t(j) * kAmKeys + 16 * lane;
            const bool wanted = lane < 8 && tok < w.hi, good = wanted && id_next >= 0 && id_next < c.pages;
            if (wanted && !good) atomicOr(a.err, kErrBadIndex);
            const int64_t id = good ? id_next : 0;
            const int64_t in_page = ((static_cast<int64_t>(w.h) << c.page_shift) + (tok & ((1 << c.page_shift) - 1))) * D;
            Place p;
            p.k = id * c.k_page + in_page;
            p.v = id * c.v_page + in_page;
            p.bytes = good ? static_cast<int>(min(w.hi - tok, int64_t(16))) * D : 0;
            p.bad = __ballot_sync(0xFFFFFFFFu, wanted && !good);
            ks = ks_next, vs = vs_next;
            ks_next = vs_next = 255;
            if (good) {
                ks_next = c.ks[id * c.ks_page + w.h];
                vs_next = c.vs[id * c.vs_page + w.h];
            }
            fetch_id(j + 1);
            return p;
        };
        bool ok = true;
        int stage = 0, issued = 0, base = 0;
        uint32_t phase = 1;
        while (ok && next_piece(a, mine, w)) {
            const int N = w.N;
            fetch_id(0);
            Place cur = place(0), next = cur;                // of the tile whose values come next, and of the one behind it
            if (N > 1) next = place(1);
            Place fetched = next;
#pragma unroll 1
            for (int item = 0; ok && item < 2 * N; ++item) {
                bool keys;
                const int j = tile_of(item, N, keys), slot = (base + j) % kAmScales;
                const bool from_cur = !keys || j == 0;
                const uint8_t* src = keys ? c.k + (from_cur ? cur.k : next.k) : c.v + cur.v;
                const int bytes = from_cur ? cur.bytes : next.bytes;
                int total = bytes;                           // of this half's four lanes
                total += __shfl_xor_sync(0xFFFFFFFFu, total, 1);
                total += __shfl_xor_sync(0xFFFFFFFFu, total, 2);
                if (keys) {
                    // Tile j's scales, before its keys: the softmax reads them with its scores. place() was last called for tile j, or
                    // at the start for tile 1. The slot's last reader was done before the keys of tile j - 1 were converted.
                    const uint32_t kb = j == 0 && N > 1 ? ks : ks_next, vb = j == 0 && N > 1 ? vs : vs_next;
                    ok = mbar_wait_warp(&raw_empty[stage], phase, abort, a.err, a.timeout_ns);
                    if (!ok) break;
                    const float e = vb == 255 ? 0.0f : static_cast<float>(static_cast<int>(vb) - 127);
                    const bool part = lane < 8 && w.from + int64_t(j) * kAmKeys + 16 * lane < w.hi;      // none behind the sequence's end
                    const uint32_t nans = __ballot_sync(0xFFFFFFFFu, part && vb == 255);
                    float2* row = scales + slot * kAmScaleRow;
                    if (lane < 8) row[lane] = make_float2(kb == 255 ? __uint_as_float(0x7FC00000u) : scale_value(kb), e);
                    if (lane == 8) row[8].x = __uint_as_float(nans);
                    if (lane == 0) bad_pages[slot] = from_cur ? cur.bad : next.bad;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&scales_full[slot]);
                }
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    ok = mbar_wait_warp(&raw_empty[stage], phase, abort, a.err, a.timeout_ns);
                    if (!ok) break;
                    if (lane == 4 * half) mbar_arrive_expect_tx(&raw_full[stage], total);
                    __syncwarp();
                    if (lane < 8 && lane >> 2 == half && bytes > 0)
                        bulk_load(smem + S::kRaw + stage * S::kHalf + (lane & 3) * 16 * D, src, bytes, &raw_full[stage]);
                    ++issued;
                    if (++stage == kAmRaw) stage = 0, phase ^= 1;
                }
                // Behind K j comes V j - 1, then K j + 1: places move on once V j - 1 is copied.
                if (keys && j > 0 && j + 1 < N) fetched = place(j + 1);
                if (!keys) {
                    cur = next;
                    next = fetched;
                }
            }
            base += N;
        }
        // No copy of this block's is left in flight when it ends.
        for (int i = max(issued - kAmRaw, 0); i < issued; ++i) mbar_wait_drain(&raw_full[i % kAmRaw], (i / kAmRaw) & 1, a.timeout_ns);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        // ---- softmax: thread = row
        const int t = warp >> 2, row = threadIdx.x & 127;
        float rowf;                                          // argument of 2^x per unit of S
        auto bring_queries = [&](const AmWork& w) {
            const int r = w.row0 + t * 128 + row;            // query row of the sequence
            const bool have = t * 128 + row < w.rows;
            const int tok = have ? a.group.div(r) : 0, head = w.h * a.G + (r - tok * a.G);
            const __nv_bfloat16* src = a.q + (w.first + tok) * a.ldq_t + head * a.ldq_h;
            uint4 x[D / 8];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) x[i] = have ? *reinterpret_cast<const uint4*>(src + i * 8) : make_uint4(0, 0, 0, 0);
            // max of both halves of every word, signs cleared
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                m = max_u16x2(m, max_u16x2(max_u16x2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu), max_u16x2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
            m = max(m & 0xFFFFu, m >> 16);
            const int E = static_cast<int>(m >> 7);
            const int up = E == 255 || m == 0 ? 0 : min(max(141 - E, -126), 126);      // as in attend_few_kernel
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            rowf = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            const uint32_t dst = smem_u32(smem) + S::kQ + t * S::kTile + row * 128;
            const uint64_t mul2 = pair(mul, mul), none = pair(-0.0f, -0.0f);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 v = unpair(fma2(pair(bf16_lo(u[k]), bf16_hi(u[k])), mul2, none));
                    o[k] = f16x2(v.x, v.y);
                }
                st_shared_v4(dst + (i >> 3) * 16384 + (((i & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[t]);
        };
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * D;
        bool ok = true;
        int base = 0, count = 0, turn = 0;                   // tiles in front; those of this half of the rows; pieces in front
        AmWork w{}, next{};
        bool more = next_piece(a, mine, w);
        if (more) bring_queries(w);
        while (ok && more) {
          more = next_piece(a, mine, next);                  // on its way while this one is worked on
          const int n = w.part[t];
          // Keys [start, stop) are seen, counted from the piece's first.
          const int r = w.row0 + t * 128 + row;
          const bool have = t * 128 + row < w.rows;
          const int tok = have ? a.group.div(r) : 0, head = w.h * a.G + (r - tok * a.G);
          const int64_t last = have ? int64_t(w.hi) - w.n + tok : -1;
          const int stop = static_cast<int>(max(last + 1 - w.from, int64_t(0))), start = static_cast<int>(max(last - a.window + 1 - w.from, int64_t(0)));
          float M = kAtNone, l = 0.0f, lift = 0.0f;            // as in attend_few_kernel
          for (int j = 0; j < n; ++j) {
            const int slot = (base + j) % kAmScales;
            // In this order: with the scores made, the scales' phase is this tile's and no earlier one's.
            ok = mbar_wait_warp(&s_full[t], (count + j) & 1, abort, a.err, a.timeout_ns) &&
                 mbar_wait_warp(&scales_full[slot], ((base + j) / kAmScales) & 1, abort, a.err, a.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            const float2* sc = scales + slot * kAmScaleRow;
            const int end = stop - j * kAmKeys, begin = start - j * kAmKeys;     // columns [begin, end) of this row are seen
            const bool masked = __any_sync(0xFFFFFFFFu, end < kAmKeys || begin > 0);
            // Half a row at a time. There is no pass for the maximum: M only has to be near enough above for f16, and the
            // sums of the weights, which are made anyway, tell whether one of them is beyond 2^15 (or l's would be beyond 2^40). If so,
            // M and lift move, O is rescaled, and the half's weights are made once more. Loops, so that the roles'
            // code stays in the instruction cache: unrolled, warps waited for instructions a fifth of the time.
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                uint32_t s[2][32];
                float* x = reinterpret_cast<float*>(s[0]);
                float most = 0.0f, sum;
                auto weights = [&]() {
                    tc_ld_32x32b_x32(ts + half * 64, s[0]);
                    tc_ld_32x32b_x32(ts + half * 64 + 32, s[1]);
                    tc_wait_ld_regs(s[0], s[1]);
                    const float least = lift - kAtLeast, above = lift + (127.0f - kAtBias), from = M - kAtBias;
                    float back[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float2 f = sc[4 * half + g];
                        const float e = fmaxf(f.y, least);
                        const float kf = f.x * rowf, d = e - from;
                        const uint64_t kf2 = pair(kf, kf), d2 = pair(d, d);
                        back[g] = pow2_biased(above - e);
#pragma unroll
                        for (int i = 16 * g; i < 16 * g + 16; i += 2) {
                            const float2 e = unpair(fma2(pair(x[i], x[i + 1]), kf2, d2));
                            x[i] = exp2_approx(e.x);
                            x[i + 1] = exp2_approx(e.y);
                        }
                    }
                    if (masked) {
                        __syncwarp();                            // a branch and not 64 selections in every tile
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t seen = seen_bits(begin, end, half * 64 + k * 32);
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[32 * k + i] = seen >> i & 1 ? x[32 * k + i] : 0.0f;
                        }
                    }
                    most = sum = 0.0f;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint64_t s0 = pair(x[16 * g], x[16 * g + 1]), s1 = pair(x[16 * g + 2], x[16 * g + 3]);
#pragma unroll
                        for (int i = 16 * g + 4; i < 16 * g + 16; i += 2) (i % 4 ? s1 : s0) = add2(i % 4 ? s1 : s0, pair(x[i], x[i + 1]));
                        const float2 r = unpair(add2(s0, s1));
                        most = fmaxf(most, r.x + r.y);
                        sum += (r.x + r.y) * back[g];
                    }
                };
                const bool begins = j + half == 0;               // M is not known
                if (!begins) weights();
                if (begins || __any_sync(0xFFFFFFFFu, most > kAmMost || sum > kAmMostSum)) {
                    float top = -INFINITY, high = -INFINITY;     // of t + e, of t
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t y[16];
                        tc_ld_32x32b_x16(ts + half * 64 + q * 16, y);
                        tc_wait_ld_regs(y);
                        const uint32_t seen = seen_bits(begin, end, half * 64 + q * 16);
                        float m = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 16; ++i) m = fmaxf(m, seen >> i & 1 ? __uint_as_float(y[i]) : -INFINITY);
                        const float2 g = sc[4 * half + q];
                        m *= g.x * rowf;
                        top = fmaxf(top, m + g.y);
                        high = fmaxf(high, m);
                    }
                    const float next = fmaxf(M, rintf(top)), f = exp2_approx(M - next);
                    const float up = next - fmaxf(M - lift, rintf(high));
                    l *= exp2_approx((M - next) - (lift - up));
                    M = next;
                    lift = up;
                    if (!begins) {                               // O, once its last product is done
                        ok = mbar_wait_warp(&o_done[2 * t + (half ^ 1)], (count + (half ? j : j - 1)) & 1, abort, a.err, a.timeout_ns);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D; q += 16) {
                            uint32_t y[16];
                            tc_ld_32x32b_x16(to + q, y);
                            tc_wait_ld_regs(y);
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                            tc_st_32x32b_x16(to + q, y);
                        }
                    }
                    weights();
                }
                uint32_t p[2][16];
#pragma unroll
                for (int i = 0; i < 64; i += 2) p[i / 32][i % 32 / 2] = f16x2(x[i], x[i + 1]);
                l += sum;
                const uint32_t nans = __float_as_uint(sc[8].x) >> 4 * half & 15;
                if (nans) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        const bool lo = half * 64 + i < end && half * 64 + i >= begin, hi = half * 64 + i + 1 < end && half * 64 + i + 1 >= begin;
                        if (nans >> i / 16 & 1) p[i / 32][i % 32 / 2] = (lo ? 0x7FFFu : 0u) | (hi ? 0x7FFF0000u : 0u);
                    }
                }
                tc_st_32x32b_x16(ts + half * 32, p[0]);          // over columns that have been read
                tc_st_32x32b_x16(ts + half * 32 + 16, p[1]);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
            }
            if (!ok) break;
        }
          if (!ok) break;
          // The next piece's queries may come once this one's are no longer read: the last scores told that, and where there were none,
          // that their barrier's phase has been seen.
          ok = mbar_wait_warp(&q_seen[t], turn & 1, abort, a.err, a.timeout_ns);
          if (!ok) break;
          ++turn;
          const int first = w.first;
          const bool whole = w.whole;
          float* part = a.many_parts + (2 * static_cast<int64_t>(blockIdx.x) + (w.begins ? 1 : 0)) * many_part_floats(D);
          base += w.N;
          count += n;
          w = next;
          if (more) bring_queries(w);
          // ---- output
          if (n > 0) {
            ok = mbar_wait_warp(&o_done[2 * t + 1], (count - 1) & 1, abort, a.err, a.timeout_ns);
            if (!ok) break;
          }
          tc_fence_after();
          const float inv = whole && l != 0.0f ? 1.0f / l : 1.0f, unit = whole ? out_unit(lift) : 1.0f;
          __nv_bfloat16* dst = a.out + (first + tok) * a.ldo_t + head * a.ldo_h;
#pragma unroll 1
          for (int q = 0; q < D; q += 32) {
            uint32_t x[32];
            if (n > 0) {
                tc_ld_32x32b_x32(to + q, x);
                tc_wait_ld_regs(x);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = n > 0 && l != 0.0f ? __float_as_uint(__uint_as_float(x[i]) * inv * unit) : 0u;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<uint4*>(part + ((q + i) / 4 * kAmRows + t * 128 + row) * 4) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            } else if (have) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(x[i + 2 * k]), __uint_as_float(x[i + 2 * k + 1]));
                        o[k] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    *reinterpret_cast<uint4*>(dst + q + i) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
          }
          if (!whole) {
            part[kAmRows * D + t * 128 + row] = M;
            part[kAmRows * D + kAmRows + t * 128 + row] = l;
            part[kAmRows * D + 2 * kAmRows + t * 128 + row] = lift;
          } else if (have && a.lse) {
            a.lse[static_cast<int64_t>(first + tok) * a.Hq + head] = l == 0.0f ? -INFINITY : (M - lift + log2f(l)) * 0.693147180559945f;
          }
          tc_fence_before();
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, kAmCols);
    if (threadIdx.x == 0 && !*abort) plan_header(a)->done[blockIdx.x] = 1;
}

// Joins the parts of units whose tiles went to several blocks (attend_many_kernel): kAmJoins blocks for every place where one block's share ends
// and the next one's begins, each with D / kAmJoins features of the unit that is cut there, if the cut is the unit's first. A
// thread per row; parts in the order of their keys.
constexpr int kAmJoins = 4;

template <int D>
__device__ __forceinline__ void join_many(const AttendArgs& a, int block) {
    const int cut = block / kAmJoins + 1, piece = block % kAmJoins, row = threadIdx.x;
    const int64_t total = plan_header(a)->total, share = many_share(a, total), x = cut * share;
    if (x >= total) return;
    const AmItem w = *plan_item(a, find_item(a, plan_header(a)->items, x));
    const int64_t cost = unit_cost(w);
    const int h = quotient(x - w.at, cost);
    const int64_t s0 = w.at + h * cost;
    if (x - s0 <= kAmUnitCost || x - share - s0 > kAmUnitCost) return;      // no tile in front of the cut, or not the first one
    const int parts = static_cast<int>((s0 + cost - 1) / share) - cut + 2;
    auto part = [&](int i) { return a.many_parts + (2 * int64_t(cut - 1 + i) + (i == 0 ? 1 : 0)) * many_part_floats(D); };
    for (int i = 0; i < parts; ++i)
        if (!plan_header(a)->done[cut - 1 + i]) return;      // a wait has run out: its rows stay as they were
    auto stat = [&](int i, int k) { return part(i)[kAmRows * D + k * kAmRows + row]; };      // M, l, lift
    float top = kAtNone, ref = kAtNone, sum = 0.0f;
    for (int i = 0; i < parts; ++i) {
        top = fmaxf(top, stat(i, 0));
        ref = fmaxf(ref, stat(i, 0) - stat(i, 2));
    }
    for (int i = 0; i < parts; ++i) sum += exp2_approx(stat(i, 0) - stat(i, 2) - ref) * stat(i, 1);
    if (row >= w.rows) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, unit = out_unit(top - ref);
    const int r = w.row0 + row, tok = a.group.div(r), head = h * a.G + (r - tok * a.G);
    __nv_bfloat16* dst = a.out + (w.first + tok) * a.ldo_t + head * a.ldo_h;
#pragma unroll
    for (int c = 0; c < D / kAmJoins; c += 8) {
        const int d = piece * (D / kAmJoins) + c;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int i = 0; i < parts; ++i) {
            const float f = exp2_approx(stat(i, 0) - top);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(part(i) + ((d / 4 + k) * kAmRows + row) * 4);
                acc[4 * k] += f * v.x, acc[4 * k + 1] += f * v.y, acc[4 * k + 2] += f * v.z, acc[4 * k + 3] += f * v.w;
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * k] * inv * unit, acc[2 * k + 1] * inv * unit);
            o[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(dst + d) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (a.lse && piece == 0)
        a.lse[static_cast<int64_t>(w.first + tok) * a.Hq + head] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.693147180559945f;
}

// `few` blocks join the parts of attend_few_kernel, the others those of attend_many_kernel.
static_assert(kAtJoinThreads == kAmRows, "a thread per row of an item");
template <int D, int NT>
__global__ void __launch_bounds__(kAtJoinThreads) attend_join_kernel(const __grid_constant__ AttendArgs a, int tiles, int few) {
    grid_wait();
    if (static_cast<int>(blockIdx.x) < few)
        join_few<D, NT>(a, tiles);
    else
        join_many<D>(a, blockIdx.x - few);
}

}  // namespace mx
