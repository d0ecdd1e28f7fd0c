// Attention over the paged E4M3 cache for many rows per sequence: prompts, and pieces of them.
//
// The mathematics is attend.cuh's; here the products decide: 4 D flops per row and key, on tcgen05. A block takes 256 query
// rows of one sequence and key head (256 / G tokens) as two tiles of 128 and walks their keys in tiles of 128:
//   S_t = Q_t K^T        tcgen05.mma kind::f16, both operands in shared memory, accumulators in TMEM
//   P_t = 2^(S_t ...)    one thread per row, read from TMEM and written back over S_t as f16
//   O_t += P_t V         P_t from TMEM, V from shared memory as it lies (features contiguous: an MN-major operand)
// While the softmax of one tile runs, the products of the other do. The codes are loaded with plain 16-byte loads, one tile ahead in
// registers, and written to shared memory as f16 (exact, one conversion for two codes): so pages may be of any size from 16 tokens and lie
// anywhere, and the scales stay out of the products: a page's key scale is a factor of the softmax's argument, its value
// scale an exponent of P, both constant over 16 columns. E4M3 operands would run at twice the rate but P (and q) would need two of them each
// to keep BF16's accuracy, which costs the softmax's threads more than the conversion costs the loaders.
//
// Roles (512 threads): warps 0-3 and 4-7 softmax of tiles 0 and 1, warps 8-11 load and convert, warp 12 issues the
// products and owns TMEM (S_0, S_1: 128 columns each, O_0, O_1: D each), warps 13-15 complete its warpgroup. The launch's 128
// registers a thread are split 192 / 80 / 40 (8 x 192 + 4 x 80 + 4 x 40 <= 16 x 128): the softmax's threads hold a row of
// scores. Every wait is bounded.
#pragma once
#include <cstdint>
#include <type_traits>

#include "attend.cuh"
#include "ptx.cuh"

namespace mx {

constexpr int kAmThreads = 512;
constexpr int kAmRows = 256;           // query rows per block
constexpr int kAmKeys = 128;           // keys per tile
constexpr int kAmRing = 2;             // stages of K and of V
constexpr int kAmScales = 4;           // tiles whose page scales are kept
constexpr uint32_t kAmCols = 512;
constexpr int kAmNoScale = -100000;    // exponent of a value scale that says NaN

template <int D>
struct AmSmem {
    static constexpr int kTile = 128 * D * 2;                      // 128 rows of f16
    static constexpr int kQ = 0;                                   // two tiles
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kAmRing * kTile;
    static constexpr int kScales = kV + kAmRing * kTile;           // [kAmScales][8] (key factor, value exponent as an integer)
    static constexpr int kBar = kScales + kAmScales * 8 * 8;
    static constexpr int kBars = 4 * kAmRing + kAmScales + 2 * 4 + 1;
    static constexpr int kMisc = kBar + kBars * 8;
    static constexpr int kBytes = kMisc + 16 + 1024;               // + alignment slack
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
// Eight products O (+)= P V of 16 keys each and the commit: P's next 16 keys lie 8 columns on, V's 2 KB on.
__device__ __forceinline__ void tc_values_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e, t, p;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t.reg .b64 b1, b2, b3, b4, b5, b6, b7;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\tadd.u32 a4, %1, 32;\n\tadd.u32 a5, %1, 40;\n\tadd.u32 a6, %1, 48;\n\tadd.u32 a7, %1, 56;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\tadd.s64 b4, %2, 512;\n\tadd.s64 b5, %2, 640;\n\tadd.s64 b6, %2, 768;\n\tadd.s64 b7, %2, 896;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar))
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

// Two fp32 lanes at once: a b + c, and a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// ---- the block's work ------------------------------------------------------------------------------------------

struct AmWork {
    int b, h, first, n, row0, rows;      // sequence, key head, its rows in the batch, the block's query rows
    int64_t hi, lo;                      // keys of the sequence; first key of the block's tiles (a multiple of 16)
    int tiles[2];                        // key tiles of either tile of rows
};

// Blocks are numbered without a prefix sum: sequence b's begin at floor(row_offsets[b] G / 256) + b, which leaves room for
// ceil(n G / 256); blocks for which nothing is left, or whose sequence has few rows, return. The last rows of a batch, which
// see the most keys, come first. By a whole warp.
__device__ __forceinline__ bool many_work(const AttendArgs& a, int block, int items, AmWork& w) {
    const CacheView& c = a.c;
    const int item = items - 1 - block / c.Hkv;
    w.h = block % c.Hkv;
    int count = 0;
    for (int b0 = 0; b0 < c.B; b0 += 32) {
        const int b = b0 + (threadIdx.x & 31);
        const int64_t at = b < c.B ? int64_t(min(max(c.row_offsets[b], 0), c.T)) * a.G / kAmRows + b : INT64_MAX;
        count += __popc(__ballot_sync(0xFFFFFFFFu, at <= item));
    }
    w.b = count - 1;
    if (w.b < 0) return false;
    rows_of(c, w.b, w.first, w.n);
    const int nth = item - static_cast<int>(int64_t(w.first) * a.G / kAmRows + w.b);
    const int64_t row0 = int64_t(nth) * kAmRows, rows = int64_t(w.n) * a.G;
    if (nth < 0 || rows <= a.most_rows || row0 >= rows) return false;
    w.row0 = static_cast<int>(row0);
    w.rows = static_cast<int>(min(rows - row0, int64_t(kAmRows)));
    w.hi = max(c.lengths[w.b], 0);
    const int64_t start = w.hi - w.n;    // position of the sequence's first row
    w.lo = max(start + a.group.div(w.row0) - a.window + 1, int64_t(0)) & ~int64_t(15);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int end = min(w.rows, (t + 1) * 128);              // rows of tiles 0 .. t
        const int64_t last = end > t * 128 ? start + a.group.div(w.row0 + end - 1) : -1;
        w.tiles[t] = last < w.lo ? 0 : static_cast<int>((last - w.lo) / kAmKeys) + 1;
    }
    return true;
}

template <int D>
__global__ void __launch_bounds__(kAmThreads, 1) attend_many_kernel(const __grid_constant__ AttendArgs a, int items) {
    grid_wait();
    using S = AmSmem<D>;
    extern __shared__ uint8_t dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kBar);
    uint64_t* k_empty = k_full + kAmRing;
    uint64_t* v_full = k_empty + kAmRing;
    uint64_t* v_empty = v_full + kAmRing;
    uint64_t* scales_full = v_empty + kAmRing;
    uint64_t* q_full = scales_full + kAmScales;
    uint64_t* s_full = q_full + 2;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 2;
    uint64_t* drain = o_done + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
    float2* scales = reinterpret_cast<float2*>(smem + S::kScales);
    const CacheView& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    AmWork w;
    if (!many_work(a, blockIdx.x, items, w)) return;       // the same in every warp
    if (threadIdx.x == 0) {
        for (int i = 0; i < kAmRing; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kAmScales; ++i) mbar_init(&scales_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
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
    const int N = max(w.tiles[0], w.tiles[1]);

    if (warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // ---- load and convert, in halves of a tile (64 keys): while one is converted the next two are on their way. Lane l < 8
        // knows where the 16 keys of group l lie, for the tile whose keys are loaded next, and hands it to the others.
        constexpr int U = 64 * D / 16 / 128;                 // 16-code pieces per thread and half tile
        constexpr int R = 2048 / D;                          // rows that the four warps take at once: 16 or 32
        const int wc = warp - 8;
        // Eight lanes: two rows and four pieces, so that their stores meet every bank once under the swizzle.
        const int row_in = wc * (R / 4) + (D == 128 ? ((lane >> 2) & 1) + 2 * (lane >> 4) : lane >> 2);
        const int piece = D == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : lane & 3;
        const int in_group = (row_in & 15) * D + piece * 16;
        int id_next = -1;                                    // page of group `lane`, of the tile behind the last one placed
        struct Places {
            int64_t k, v;                                    // of group `lane`: bytes from the codes' beginning
            int valid;                                       // its keys; 0 outside the sequence or on a bad page
            uint32_t scales;
        };
        auto fetch_id = [&](int j) {
            const int64_t tok = w.lo + int64_t(j) * kAmKeys + 16 * lane;
            id_next = -1;
            if (lane < 8 && j < N && tok < w.hi) {
                id_next = static_cast<int>(page_id(c, w.b, tok >> c.page_shift));
                if (id_next < 0) atomicOr(a.err, kErrBadIndex);
            }
        };
        auto place = [&](int j) {                            // from id_next; then fetches the next tile's
            Places p;
            const int64_t tok = w.lo + int64_t(j) * kAmKeys + 16 * lane;
            const int64_t in_page = ((static_cast<int64_t>(w.h) << c.page_shift) + (tok & ((1 << c.page_shift) - 1))) * D;
            p.valid = id_next < 0 ? 0 : static_cast<int>(min(w.hi - tok, int64_t(16)));
            p.k = id_next * c.k_page + in_page;
            p.v = id_next * c.v_page + in_page;
            p.scales = id_next < 0 ? 0xFFFFu : c.ks[id_next * c.ks_page + w.h] | static_cast<uint32_t>(c.vs[id_next * c.vs_page + w.h]) << 8;
            fetch_id(j + 1);
            return p;
        };
        auto load = [&](const uint8_t* base, int64_t of_group, int valid, int half, uint4 (&x)[U]) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int group = half * 4 + (i * R + row_in) / 16;
                const int64_t at = __shfl_sync(0xFFFFFFFFu, of_group, group);
                const int rows = __shfl_sync(0xFFFFFFFFu, valid, group);
                x[i] = make_uint4(0, 0, 0, 0);
                if ((row_in & 15) < rows) x[i] = ld_once_v4(base + at + in_group);
            }
        };
        auto convert = [&](uint32_t tile, int half, const uint4 (&x)[U]) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int row = half * 64 + i * R + row_in;
                const uint32_t at = tile + (piece >> 2) * 16384 + row * 128, c0 = (piece & 3) * 2, sw = row & 7;
                st_shared_v4(at + ((c0 ^ sw) << 4), f16x2_of_e4m3(x[i].x), f16x2_of_e4m3_hi(x[i].x), f16x2_of_e4m3(x[i].y), f16x2_of_e4m3_hi(x[i].y));
                st_shared_v4(at + (((c0 + 1) ^ sw) << 4), f16x2_of_e4m3(x[i].z), f16x2_of_e4m3_hi(x[i].z), f16x2_of_e4m3(x[i].w), f16x2_of_e4m3_hi(x[i].w));
            }
        };
        uint4 x0[U], x1[U];                                  // the two halves that are converted next
        // Converts them into `tile` and loads the halves of the tile behind it if there is `more`.
        auto pass_on = [&](uint32_t tile, bool more, const uint8_t* base, int64_t of_group, int valid) {
            convert(tile, 0, x0);
            if (more) load(base, of_group, valid, 0, x0);
            convert(tile, 1, x1);
            if (more) load(base, of_group, valid, 1, x1);
            fence_async_smem();
            __syncwarp();
        };
        auto keys = [&](int j, const Places& p) {            // room for tile j's keys, and its scales
            if (wc == 0 && lane < 8) {
                const uint32_t kb = p.scales & 0xFFu, vb = p.scales >> 8;
                scales[(j % kAmScales) * 8 + lane] = make_float2(kb == 255 ? __uint_as_float(0x7FC00000u) : scale_value(kb),
                                                                 __int_as_float(vb == 255 ? kAmNoScale : static_cast<int>(vb) - 127));
            }
            return j < kAmRing || mbar_wait_warp(&k_empty[j % kAmRing], (j / kAmRing - 1) & 1, abort, a.err, a.timeout_ns);
        };
        auto keys_done = [&](int j) {
            if (lane == 0) {
                mbar_arrive(&k_full[j % kAmRing]);
                if (wc == 0) mbar_arrive(&scales_full[j % kAmScales]);
            }
        };
        // Order of the tiles: K 0, then K j + 1 and V j for j = 0, 1, ...
        if (N > 0) {
            const uint32_t kt = smem_u32(smem) + S::kK, vt = smem_u32(smem) + S::kV;
            fetch_id(0);
            Places cur = place(0), next = cur;
            load(c.k, cur.k, cur.valid, 0, x0);
            load(c.k, cur.k, cur.valid, 1, x1);
            if (N > 1) next = place(1);
            bool ok = keys(0, cur);
            pass_on(kt, true, N > 1 ? c.k : c.v, N > 1 ? next.k : cur.v, N > 1 ? next.valid : cur.valid);
            keys_done(0);
            for (int j = 0; ok && j < N; ++j) {
                if (j + 1 < N) {
                    ok = keys(j + 1, next);
                    if (!ok) break;
                    pass_on(kt + (j + 1) % kAmRing * S::kTile, true, c.v, cur.v, cur.valid);
                    keys_done(j + 1);
                }
                Places after = next;
                if (j + 2 < N) after = place(j + 2);
                if (j >= kAmRing) ok = mbar_wait_warp(&v_empty[j % kAmRing], (j / kAmRing - 1) & 1, abort, a.err, a.timeout_ns);
                if (!ok) break;
                pass_on(vt + j % kAmRing * S::kTile, j + 1 < N, j + 2 < N ? c.k : c.v, j + 2 < N ? after.k : next.v, after.valid);
                if (lane == 0) mbar_arrive(&v_full[j % kAmRing]);
                cur = next;
                next = after;
            }
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 12) {
        // ---- products
        constexpr uint32_t idesc_s = idesc_f16(128, kAmKeys, false), idesc_o = idesc_f16(128, D, true);
        const uint32_t base = smem_u32(smem);
        const uint64_t q_desc = sdesc_kmajor_sw128(base + S::kQ), k_desc = sdesc_kmajor_sw128(base + S::kK), v_desc = sdesc_mnmajor_sw128(base + S::kV);
        auto scores = [&](int t, int st) {
            tc_scores_elect<D>(tmem + t * 128, q_desc + t * (S::kTile >> 4), k_desc + st * (S::kTile >> 4), idesc_s, &s_full[t]);
        };
        bool ok = true;
        if (N > 0) {
            ok = mbar_wait_warp(&q_full[0], 0, abort, a.err, a.timeout_ns) && mbar_wait_warp(&q_full[1], 0, abort, a.err, a.timeout_ns) &&
                 mbar_wait_warp(&k_full[0], 0, abort, a.err, a.timeout_ns);
            if (ok) {
                tc_fence_after();
                for (int t = 0; t < 2; ++t)
                    if (w.tiles[t] > 0) scores(t, 0);
                tc_commit_elect(&k_empty[0]);
            }
        }
        for (int j = 0; ok && j < N; ++j) {
            const int vs = j % kAmRing, kn = (j + 1) % kAmRing;
            ok = mbar_wait_warp(&v_full[vs], (j / kAmRing) & 1, abort, a.err, a.timeout_ns);
            if (!ok) break;
            bool have_k = false;
            for (int t = 0; t < 2; ++t) {
                if (j < w.tiles[t]) {
                    ok = mbar_wait_warp(&p_full[t], j & 1, abort, a.err, a.timeout_ns);
                    if (!ok) break;
                    tc_fence_after();
                    tc_values_elect(tmem + 256 + t * D, tmem + t * 128, v_desc + vs * (S::kTile >> 4), idesc_o, j != 0, &o_done[t]);
                }
                if (j + 1 < w.tiles[t]) {
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
        // Every product issued by this warp has completed once `drain` fires.
        tc_commit_elect(drain);
        mbar_wait_drain(drain, 0, a.timeout_ns);
        __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // ---- softmax: thread = row
        const int t = warp >> 2, row = threadIdx.x & 127;
        const int r = w.row0 + t * 128 + row;                // query row of the sequence
        const bool have = t * 128 + row < w.rows;
        const int tok = have ? a.group.div(r) : 0, head = w.h * a.G + (r - tok * a.G);
        float rowf;
        {
            const __nv_bfloat16* src = a.q + (w.first + tok) * a.ldq_t + head * a.ldq_h;
            uint4 x[D / 8];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                x[i] = have ? *reinterpret_cast<const uint4*>(src + i * 8) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) m = max(m, max(u[k] & 0x7FFFu, (u[k] >> 16) & 0x7FFFu));
            }
            const int E = static_cast<int>(m >> 7);
            const int up = E == 255 || m == 0 ? 0 : min(max(141 - E, -126), 126);      // as in attend_few_kernel
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            rowf = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            const uint32_t dst = smem_u32(smem) + S::kQ + t * S::kTile + row * 128;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = f16x2(bf16_lo(u[k]) * mul, bf16_hi(u[k]) * mul);
                st_shared_v4(dst + (i >> 3) * 16384 + (((i & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[t]);
        }
        const int64_t last = have ? w.hi - w.n + tok : -1, from = last - a.window + 1;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * D;
        float M = kAtNone, l = 0.0f;
        int E = kAmNoScale;
        const int n = w.tiles[t];
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = mbar_wait_warp(&scales_full[j % kAmScales], (j / kAmScales) & 1, abort, a.err, a.timeout_ns) &&
                 mbar_wait_warp(&s_full[t], j & 1, abort, a.err, a.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            const float2* sc = scales + (j % kAmScales) * 8;
            const int64_t key0 = w.lo + int64_t(j) * kAmKeys;
            // Columns [begin, end) of this row are seen.
            const int end = static_cast<int>(min(max(last + 1 - key0, int64_t(0)), int64_t(kAmKeys)));
            const int begin = static_cast<int>(min(max(from - key0, int64_t(0)), int64_t(kAmKeys)));
            const bool masked = __any_sync(0xFFFFFFFFu, end < kAmKeys || begin > 0);
            // MASKED as a type: the unmasked tiles, nearly all, have no trace of the mask in their code.
            float s[kAmKeys];
            float top = -INFINITY;
            int ev = kAmNoScale;
            auto read = [&](auto MASKED) {
                uint32_t(&u)[kAmKeys] = reinterpret_cast<uint32_t(&)[kAmKeys]>(s);
#pragma unroll
                for (int q = 0; q < 4; ++q) tc_ld_32x32b_x32(ts + q * 32, reinterpret_cast<uint32_t(&)[32]>(u[32 * q]));
                tc_wait_ld_regs(u);
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if constexpr (MASKED.value)
#pragma unroll
                        for (int i = 16 * g; i < 16 * g + 16; ++i)
                            if (i >= end || i < begin) s[i] = -INFINITY;
                    float m = fmaxf(s[16 * g], s[16 * g + 1]);
#pragma unroll
                    for (int i = 2; i < 16; i += 2) m = fmaxf(m, fmaxf(s[16 * g + i], s[16 * g + i + 1]));
                    const float2 f = sc[g];
                    top = fmaxf(top, m * (f.x * rowf));
                    ev = max(ev, __float_as_int(f.y));
                }
            };
            if (masked)
                read(std::true_type());
            else
                read(std::false_type());
            const bool grown = ev > E;                       // the same in every row
            if (__any_sync(0xFFFFFFFFu, top > M + kAtSlack) || grown) {
                const float next = fmaxf(M, top);
                const float f = exp2_approx(M - next), fo = grown ? ldexpf(f, max(E - ev, -300)) : f;
                M = next;
                l *= f;
                if (grown) E = ev;
                if (j > 0) {                                 // O, once its last product is done
                    ok = mbar_wait_warp(&o_done[t], (j - 1) & 1, abort, a.err, a.timeout_ns);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < D; q += 16) {
                        uint32_t x[16];
                        tc_ld_32x32b_x16(to + q, x);
                        tc_wait_ld_regs(x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fo);
                        tc_st_32x32b_x16(to + q, x);
                    }
                }
            }
            // P, and the weights left in s for the sum, which is made once the products have theirs.
            auto weights = [&](auto MASKED) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t p[16];
#pragma unroll
                    for (int g = 2 * q; g < 2 * q + 2; ++g) {
                        const float2 f = sc[g];
                        const int dv = __float_as_int(f.y) - E;
                        const bool apart = dv < -kAtValueRange;          // values that do not count, or that are NaN
                        const float kf = f.x * rowf, d = static_cast<float>(kAtBias + (apart ? 0 : dv)) - M;
                        uint32_t seen = 0xFFFFu;
#pragma unroll
                        for (int i = 16 * g; i < 16 * g + 16; i += 2) {
                            const bool none0 = MASKED.value && s[i] == -INFINITY, none1 = MASKED.value && s[i + 1] == -INFINITY;
                            float2 x = fma2(make_float2(s[i], s[i + 1]), make_float2(kf, kf), make_float2(d, d));
                            s[i] = none0 ? 0.0f : exp2_approx(x.x);
                            s[i + 1] = none1 ? 0.0f : exp2_approx(x.y);
                            if (MASKED.value && apart) seen &= ~((none0 ? 1u : 0u) << (i % 16) | (none1 ? 2u : 0u) << (i % 16));
                            p[(i / 2) % 16] = f16x2(s[i], s[i + 1]);
                        }
                        if (apart) {
                            const bool nan = __float_as_int(f.y) == kAmNoScale;
#pragma unroll
                            for (int i = 0; i < 16; i += 2)
                                p[(8 * g + i / 2) % 16] = nan ? (seen >> i & 1 ? 0x7FFFu : 0u) | (seen >> i & 2 ? 0x7FFF0000u : 0u) : 0u;
                        }
                    }
                    tc_st_32x32b_x16(ts + q * 16, p);
                }
            };
            if (masked)
                weights(std::true_type());
            else
                weights(std::false_type());
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[t]);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int dv = __float_as_int(sc[g].y) - E, shift = kAtBias + (dv < -kAtValueRange ? 0 : dv);
                float2 sum = make_float2(s[16 * g], s[16 * g + 1]);
#pragma unroll
                for (int i = 16 * g + 2; i < 16 * g + 16; i += 2) sum = add2(sum, make_float2(s[i], s[i + 1]));
                l += (sum.x + sum.y) * __int_as_float((127 - shift) << 23);
            }
        }
        // ---- output
        if (ok && n > 0) ok = mbar_wait_warp(&o_done[t], (n - 1) & 1, abort, a.err, a.timeout_ns);
        if (ok) {
            tc_fence_after();
            const float inv = l == 0.0f ? 0.0f : ldexpf(1.0f / l, E - kAtBias);
            __nv_bfloat16* dst = a.out + (w.first + tok) * a.ldo_t + head * a.ldo_h;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t x[32];
                if (n > 0) {
                    tc_ld_32x32b_x32(to + q * 32, x);
                    tc_wait_ld_regs(x);
                }
                if (!have) continue;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(x[i + 2 * k]) * inv, __uint_as_float(x[i + 2 * k + 1]) * inv);
                        o[k] = n > 0 && l != 0.0f ? *reinterpret_cast<const uint32_t*>(&v) : 0u;
                    }
                    *reinterpret_cast<uint4*>(dst + q * 32 + i) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (have && a.lse)
                a.lse[static_cast<int64_t>(w.first + tok) * a.Hq + head] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.693147180559945f;
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, kAmCols);
}

}  // namespace mx
