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
// Roles (416 threads): warps 0-3 and 4-7 softmax of tiles 0 and 1, warps 8-11 load and convert, warp 12 issues the
// products and owns TMEM (S_0, S_1: 128 columns each, O_0, O_1: D each). Every wait is bounded.
#pragma once
#include <cstdint>

#include "attend.cuh"
#include "ptx.cuh"

namespace mx {

constexpr int kAmThreads = 416;
constexpr int kAmRows = 256;           // query rows per block
constexpr int kAmKeys = 128;           // keys per tile
constexpr int kAmRing = 2;             // stages of K and of V
constexpr int kAmScales = 4;           // tiles whose page scales are kept
constexpr uint32_t kAmCols = 512;

template <int D>
struct AmSmem {
    static constexpr int kTile = 128 * D * 2;                      // 128 rows of f16
    static constexpr int kQ = 0;                                   // two tiles
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kAmRing * kTile;
    static constexpr int kScales = kV + kAmRing * kTile;           // [kAmScales][8] (key factor, value exponent)
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
__device__ __forceinline__ void tc_mma_f16_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void tc_mma_f16_tmem_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
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
__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
        // ---- load and convert. A warp's unit i is four (D = 128) or eight (D = 64) rows of 16-row group(s); lane l < 8
        // keeps the page of group l.
        constexpr int U = 128 * D / 16 / 128;               // 16-code pieces per thread and tile
        const int wc = warp - 8;
        const int rl = D == 128 ? ((lane >> 2) & 1) + 2 * (lane >> 4) : lane >> 2;      // row within the warp's rows of a unit
        const int piece = D == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : lane & 3;
        constexpr int R = 2048 / D;                          // rows of a unit over the four warps: 16 or 32
        const int row_in = wc * (R / 4) + rl;
        int64_t id_next = -1, id_cur = -1, id_v = -1;        // page of group `lane` of the tiles whose keys are loaded next, last, whose values are
        auto fetch_ids = [&](int j) {
            const int64_t tok = w.lo + int64_t(j) * kAmKeys + 16 * lane;
            id_next = -1;
            if (lane < 8 && j < N && tok < w.hi) {
                id_next = page_id(c, w.b, tok >> c.page_shift);
                if (id_next < 0) atomicOr(a.err, kErrBadIndex);
            }
        };
        auto load = [&](const uint8_t* base, int64_t stride, int64_t ids, int j, uint4 (&x)[U]) {
            const int64_t key0 = w.lo + int64_t(j) * kAmKeys;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int row = i * R + row_in;
                const int64_t tok = key0 + row;
                const int64_t id = __shfl_sync(0xFFFFFFFFu, ids, row >> 4);
                x[i] = make_uint4(0, 0, 0, 0);
                if (id >= 0 && tok < w.hi)
                    x[i] = ld_once_v4(base + id * stride +
                                      (((static_cast<int64_t>(w.h) << c.page_shift) + (tok & ((1 << c.page_shift) - 1))) * D + piece * 16));
            }
        };
        auto convert = [&](uint32_t tile, const uint4 (&x)[U]) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int row = i * R + row_in;
                const uint32_t at = tile + (piece >> 2) * 16384 + row * 128, c0 = (piece & 3) * 2, sw = row & 7;
                st_shared_v4(at + ((c0 ^ sw) << 4), f16x2_of_e4m3(x[i].x), f16x2_of_e4m3_hi(x[i].x), f16x2_of_e4m3(x[i].y), f16x2_of_e4m3_hi(x[i].y));
                st_shared_v4(at + (((c0 + 1) ^ sw) << 4), f16x2_of_e4m3(x[i].z), f16x2_of_e4m3_hi(x[i].z), f16x2_of_e4m3(x[i].w), f16x2_of_e4m3_hi(x[i].w));
            }
            fence_async_smem();
            __syncwarp();
        };
        uint4 kx[U], vx[U];
        bool ok = true;
        fetch_ids(0);
        id_cur = id_next;
        load(c.k, c.k_page, id_cur, 0, kx);
        // Order of the tiles: K 0, then K j + 1 and V j for j = 0, 1, ...
        for (int j = -1; ok && j < N; ++j) {
            const int jk = j + 1;
            if (jk < N) {
                fetch_ids(jk + 1);
                // Scales of tile jk, before its keys: the softmax reads them with its scores.
                if (wc == 0) {
                    float2 s = make_float2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
                    if (lane < 8 && id_cur >= 0) {
                        const uint32_t kb = c.ks[id_cur * c.ks_page + w.h], vb = c.vs[id_cur * c.vs_page + w.h];
                        if (kb != 255) s.x = scale_value(kb);
                        if (vb != 255) s.y = static_cast<float>(static_cast<int>(vb) - 127);
                    }
                    if (lane < 8) scales[(jk % kAmScales) * 8 + lane] = s;
                }
                const int st = jk % kAmRing;
                if (jk >= kAmRing) ok = mbar_wait_warp(&k_empty[st], (jk / kAmRing - 1) & 1, abort, a.err, a.timeout_ns);
                if (!ok) break;
                convert(smem_u32(smem) + S::kK + st * S::kTile, kx);
                if (lane == 0) {
                    mbar_arrive(&k_full[st]);
                    if (wc == 0) mbar_arrive(&scales_full[jk % kAmScales]);
                }
                id_v = id_cur;
                id_cur = id_next;
                if (jk + 1 < N) load(c.k, c.k_page, id_cur, jk + 1, kx);
            }
            if (j >= 0) {
                const int st = j % kAmRing;
                if (j >= kAmRing) ok = mbar_wait_warp(&v_empty[st], (j / kAmRing - 1) & 1, abort, a.err, a.timeout_ns);
                if (!ok) break;
                convert(smem_u32(smem) + S::kV + st * S::kTile, vx);
                if (lane == 0) mbar_arrive(&v_full[st]);
            }
            if (jk < N) load(c.v, c.v_page, id_v, jk, vx);
        }
    } else if (warp == 12) {
        // ---- products
        constexpr uint32_t idesc_s = idesc_f16(128, kAmKeys, false), idesc_o = idesc_f16(128, D, true);
        const uint32_t base = smem_u32(smem);
        auto scores = [&](int t, int st) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
                tc_mma_f16_elect(tmem + t * 128, sdesc_kmajor_sw128(base + S::kQ + t * S::kTile + off),
                                 sdesc_kmajor_sw128(base + S::kK + st * S::kTile + off), idesc_s, k != 0);
            }
            tc_commit_elect(&s_full[t]);
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
#pragma unroll
                    for (int k = 0; k < kAmKeys / 16; ++k)
                        tc_mma_f16_tmem_elect(tmem + 256 + t * D, tmem + t * 128 + k * 8,
                                              sdesc_mnmajor_sw128(base + S::kV + vs * S::kTile + k * 2048), idesc_o, j != 0 || k != 0);
                    tc_commit_elect(&o_done[t]);
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
    } else if (warp < 8) {
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
        int E = -1000;
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
            float top = -INFINITY;
            int ev = -1000;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t s[32];
                tc_ld_32x32b_x32(ts + q * 32, s);
                tc_wait_ld_regs(s);
                if (masked)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (q * 32 + i >= end || q * 32 + i < begin) s[i] = 0xFF800000u;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float m = fmaxf(__uint_as_float(s[16 * g]), __uint_as_float(s[16 * g + 1]));
#pragma unroll
                    for (int i = 2; i < 16; i += 2) m = fmaxf(m, fmaxf(__uint_as_float(s[16 * g + i]), __uint_as_float(s[16 * g + i + 1])));
                    const float2 f = sc[2 * q + g];
                    top = fmaxf(top, m * (f.x * rowf));
                    if (f.y == f.y) ev = max(ev, static_cast<int>(f.y));
                }
            }
            const bool grown = ev > E;                       // the same in every row
            if (__any_sync(0xFFFFFFFFu, top > M + kAtSlack) || grown) {
                const float next = fmaxf(M, top);
                const float f = exp2_approx(M - next), fo = grown ? ldexpf(f, max(E - ev, -200)) : f;
                M = next;
                l *= f;
                if (grown) E = ev;
                if (j > 0) {                                 // O, once its last product is done
                    ok = mbar_wait_warp(&o_done[t], (j - 1) & 1, abort, a.err, a.timeout_ns);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t x[32];
                        tc_ld_32x32b_x32(to + q * 32, x);
                        tc_wait_ld_regs(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fo);
                        tc_st_32x32b_x32(to + q * 32, x);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t s[32], p[16];
                tc_ld_32x32b_x32(ts + q * 32, s);
                tc_wait_ld_regs(s);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float2 f = sc[2 * q + g];
                    const int dv = f.y == f.y ? static_cast<int>(f.y) - E : 0;
                    const bool apart = f.y != f.y || dv < -kAtValueRange;
                    const float shift = kAtBias + static_cast<float>(apart ? 0 : dv), kf = f.x * rowf, d = shift - M;
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float2 x = fma2(make_float2(__uint_as_float(s[16 * g + i]), __uint_as_float(s[16 * g + i + 1])), make_float2(kf, kf), make_float2(d, d));
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        if (masked) {
                            const int col = q * 32 + 16 * g + i;
                            if (col >= end || col < begin) x.x = 0.0f;
                            if (col + 1 >= end || col + 1 < begin) x.y = 0.0f;
                        }
                        sum = add2(sum, x);
                        p[8 * g + i / 2] = f16x2(x.x, x.y);
                    }
                    l += (sum.x + sum.y) * exp2_approx(-shift);
                    if (apart) {                             // values that do not count, or that are NaN
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const int col = q * 32 + 16 * g + i;
                            const bool none = f.y == f.y;
                            const uint32_t lo = none || col >= end || col < begin ? 0u : 0x7FFFu;
                            const uint32_t hi = none || col + 1 >= end || col + 1 < begin ? 0u : 0x7FFF0000u;
                            p[8 * g + i / 2] = lo | hi;
                        }
                    }
                }
                tc_st_32x32b_x16(ts + q * 16, p);            // over columns that have been read
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[t]);
        }
        // ---- output
        if (ok && n > 0) ok = mbar_wait_warp(&o_done[t], (n - 1) & 1, abort, a.err, a.timeout_ns);
        if (ok) {
            tc_fence_after();
            const float inv = l == 0.0f ? 0.0f : ldexpf(1.0f / l, E - static_cast<int>(kAtBias));
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
