// MXFP4 product for few rows of A (at most 32, up to 64 for a long K: the tokens of a decoding step), bound by one pass
// over the weight.
//
// C[m, n] = sum_k A[m, k] B[n, k] is computed as its transpose: 128 rows of the weight B are the tensor core's 128
// rows and the tokens its columns (NPAD = 16, 32 or 64 of them), so no lane of the MMA works on padding and a CTA's
// loads are almost all weight bytes. The CTA-pair kernel's 256 x 256 tiles would leave two thirds of the SMs without
// work at N = 6144 and fill its A tiles with zeros.
//
// K is split over the CTAs of a cluster (1, 2, 4 or 8), as many as keep every SM busy: CTA r takes a contiguous share
// of the 256-element stages, its fp32 accumulator goes to its shared memory, and after a cluster barrier each CTA sums
// 128 / cluster columns of C over all of them in rank order through distributed shared memory, so neither a workspace
// nor atomics are needed and the result does not depend on timing.
//
// Roles (192 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA issuer, warps 2-5 epilogue. Four stages of at
// most 26 KB, two CTAs per SM, so up to 130 KB of weight are in flight per SM. Waits are bounded as in the other
// kernels; no load uses cluster multicast.
//
// Measured with weights that are not in L2 (a graph over up to 20 of them), this kernel / the pair kernel in us: 16 x 6144 x
// 4096 8.2 / 11.8 (13.4 MB), 16 x 24576 x 4096 13.6 / 20.2, 16 x 151936 x 4096 59 / 77 (5.6 TB/s), 32 x 2048 x 1024
// 6.6 / 7.0. The smallest call takes 3.3 us: launch, tensor maps, one load, one MMA.
#pragma once
#include <cstdint>

#include "gemm.cuh"

namespace mx {

// Up to 32 rows this kernel is the faster one but for weights of many short rows (N >= 40960, K <= 1024: up to 1.8 times the
// pair kernel's time at 151936 x 256). 33 to 64 rows take its widest form, whose fixed part is larger; this kernel /
// the pair kernel in us at 64 rows:
//   K        256          1024         2048         4096         8192
//   N 512    7.8 / 5.9    8.8 / 7.2    8.4 / 8.6    8.8 / 10.6   9.4 / 15.1
//   N 8192   7.9 / 6.1    9.6 / 7.6    10.4 / 9.6   12.3 / 12.5  14.6 / 17.3
//   N 24576  8.8 / 7.4    11.5 / 11.1  13.3 / 13.9  18.1 / 19.8  26.2 / 30.9
//   N 40960  15.4 / 8.4   19.0 / 12.9  23.2 / 17.8  31.9 / 26.4  48.3 / 44.1
constexpr int kFewRows = 32;
constexpr int kFewMaxRows = 64;
constexpr int kFewLongK = 4096;                 // from here on also for 33 to 64 rows
constexpr int kFewThreads = 192;
constexpr int kFewStages = 4;
constexpr int kFewSf = 1024;                    // two 512-byte scale blocks per operand and stage

template <int NPAD>
struct FewSmem {
    static constexpr int kA = 0;                                        // weight tiles, 128 rows x 128 bytes
    static constexpr int kB = kA + kFewStages * 128 * 128;              // token tiles, NPAD rows x 128 bytes
    static constexpr int kSfa = kB + kFewStages * NPAD * 128;
    static constexpr int kSfb = kSfa + kFewStages * kFewSf;
    static constexpr int kBar = kSfb + kFewStages * kFewSf;
    static constexpr int kMisc = kBar + (2 * kFewStages + 1) * 8;
    static constexpr int kBytes = kMisc + 16 + 1024;                    // + alignment slack
    static constexpr uint32_t kStageBytes = 128 * 128 + NPAD * 128 + 2 * kFewSf;
    static_assert(NPAD * 128 * 4 <= kFewStages * 128 * 128, "the partial sums reuse the weight tiles");
};

struct FewArgs {
    void* c;
    int64_t ldc;
    int M, N, K;
    int nkb;                 // stages of 256 elements of K
    int out_bf16;
    uint32_t* err;
    uint64_t timeout_ns;
};

__device__ __forceinline__ float4 ld_shared_cluster_f32x4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

template <int NPAD>
__global__ void __launch_bounds__(kFewThreads, 2)
    mx_gemm_fp4_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                           const __grid_constant__ CUtensorMap tmap_sfw, const __grid_constant__ CUtensorMap tmap_sfx,
                           const FewArgs a) {
    using L = FewSmem<NPAD>;
    constexpr int S = kFewStages;
    constexpr uint32_t kCols = 128;             // TMEM: NPAD accumulator columns, then two scale slots of 8
    constexpr uint32_t kSf = 64;
    grid_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int tile = static_cast<int>(blockIdx.x) / ranks;
    const int n0 = tile * 128;
    const int kb_begin = a.nkb * rank / ranks, kb_end = a.nkb * (rank + 1) / ranks;

    auto load = [&](int kb, int stage) {
        mbar_arrive_expect_tx_elect(&full[stage], L::kStageBytes);
        tma_load_2d_elect(smem + L::kA + stage * 128 * 128, &tmap_w, &full[stage], kb * kBK, n0);
        tma_load_2d_elect(smem + L::kB + stage * NPAD * 128, &tmap_x, &full[stage], kb * kBK, 0);
        tma_load_3d_elect(smem + L::kSfa + stage * kFewSf, &tmap_sfw, &full[stage], 0, 4 * kb, tile);
        tma_load_3d_elect(smem + L::kSfb + stage * kFewSf, &tmap_sfx, &full[stage], 0, 4 * kb, 0);
    };
    const int ahead = min(S, kb_end - kb_begin);
    if (warp == 0) {
        if (lane == 0) {
            for (int s = 0; s < S; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            mbar_init(done, 1);
            *abort = 0;
            fence_barrier_init();
        }
        __syncwarp();
        // The first stages' loads start before the rest of the CTA is set up.
        for (int i = 0; i < ahead; ++i) load(kb_begin + i, i);
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_base_slot;

    if (warp == 0) {
        int stage = ahead % S, issued = ahead;
        uint32_t phase = ahead / S;
        for (int kb = kb_begin + ahead; kb < kb_end; ++kb) {
            if (!mbar_wait_warp(&empty[stage], phase ^ 1u, abort, a.err, a.timeout_ns)) break;
            load(kb, stage);
            ++issued;
            if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        // No copy may be in flight when the CTA leaves, whatever the other roles did: wait for the last
        // min(issued, S) fills.
        int s = stage;
        uint32_t p = phase;
        for (int i = 0; i < min(issued, S); ++i) {
            if (--s < 0) { s = S - 1; p ^= 1u; }
            mbar_wait_drain(&full[s], p, a.timeout_ns);
        }
    } else if (warp == 1) {
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = kb_begin; kb < kb_end; ++kb) {
            if (!mbar_wait_warp(&full[stage], phase, abort, a.err, a.timeout_ns)) break;
            tc_fence_after();
            const uint64_t adesc = sdesc_kmajor_sw128(smem_u32(smem + L::kA + stage * 128 * 128));
            const uint64_t bdesc = sdesc_kmajor_sw128(smem_u32(smem + L::kB + stage * NPAD * 128));
            const uint64_t sda = sdesc_scale_block(smem_u32(smem + L::kSfa + stage * kFewSf));
            const uint64_t sdb = sdesc_scale_block(smem_u32(smem + L::kSfb + stage * kFewSf));
            const int left = a.K - kb * 256;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sfa_t = tmem_base + kSf + 8u * h, sfb_t = sfa_t + 4u;
                tc_cp_elect(sfa_t, sda + 32u * h);
                tc_cp_elect(sfb_t, sdb + 32u * h);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // K-step k: +32 bytes (64 elements); scale slot k / 2, scale bytes 2 (k % 2), +1 of the word.
                const uint32_t id = 2u * (k & 1), sfa_t = tmem_base + kSf + 8u * (k >> 1);
                if (64 * k < left)
                    tc_mma_mxf4_elect(tmem_base, adesc + 2u * k, bdesc + 2u * k, idesc_mxf4(128, NPAD, id),
                                      sfa_t | (id << 30), (sfa_t + 4u) | (id << 30), (kb != kb_begin || k != 0) ? 1u : 0u);
            }
            tc_commit_elect(&empty[stage]);
            if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        // Every MMA issued by this warp has completed once `done` fires; the epilogue waits for it too.
        __syncwarp();
        tc_commit_elect(done);
        mbar_wait_drain(done, 0, a.timeout_ns);
    } else {
        // The accumulator: lane l of quadrant q is weight row 32 q + l, column m token m.
        const int q = warp & 3;
        const int n = n0 + 32 * q + lane;
        // `done` fires too when the issuer has given up: what it had accumulated until then is no result.
        const bool ok = mbar_wait_warp(done, 0, abort, a.err, a.timeout_ns) && __all_sync(0xFFFFFFFFu, !*abort);
        tc_fence_after();
        float* part = reinterpret_cast<float*>(smem + L::kA);            // [NPAD][128]
        if (ok) {
#pragma unroll
            for (int m0 = 0; m0 < NPAD; m0 += 16) {
                uint32_t r[16];
                tc_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + m0, r);
                tc_wait_ld_regs(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int m = m0 + i;
                    if (ranks > 1) {
                        part[m * 128 + 32 * q + lane] = __uint_as_float(r[i]);
                    } else if (m < a.M && n < a.N) {
                        if (a.out_bf16)
                            static_cast<__nv_bfloat16*>(a.c)[m * a.ldc + n] = __float2bfloat16_rn(__uint_as_float(r[i]));
                        else
                            static_cast<float*>(a.c)[m * a.ldc + n] = __uint_as_float(r[i]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (ranks > 1) {
        cluster_sync();                         // every CTA's partial sums are in its shared memory
        // No CTA writes sums of which another one, whose wait has run out, did not deliver its part.
        const uint32_t gave_up = ld_shared_cluster_u32(mapa_shared(smem_u32(smem + L::kMisc + 4), lane & (ranks - 1)));
        if (warp >= 2 && __all_sync(0xFFFFFFFFu, gave_up == 0)) {
            // Four consecutive columns per thread; width / 4 (a power of two) threads per row.
            const int width = 128 / ranks, per_row = width / 4, t = threadIdx.x - 64;
            const uint32_t part = smem_u32(smem + L::kA);
            const int nl = rank * width + 4 * (t & (per_row - 1));
            const int n = n0 + nl;
            for (int m = t / per_row; m < a.M; m += 128 / per_row) {
                float4 v[8], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < ranks) v[r] = ld_shared_cluster_f32x4(mapa_shared(part + (m * 128 + nl) * 4, r));
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < ranks) {
                        sum.x += v[r].x;
                        sum.y += v[r].y;
                        sum.z += v[r].z;
                        sum.w += v[r].w;
                    }
                const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.N) {
                        if (a.out_bf16)
                            static_cast<__nv_bfloat16*>(a.c)[m * a.ldc + n + i] = __float2bfloat16_rn(out[i]);
                        else
                            static_cast<float*>(a.c)[m * a.ldc + n + i] = out[i];
                    }
            }
        }
        cluster_sync();                         // no CTA leaves while another reads its shared memory
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kCols);
    }
}

// ---- grouped: a decoding step of an MoE layer ------------------------------------------------------------
//
// The same transposed tiles for experts of a few rows each, where the CTA-pair kernel's 256 x 256 tiles compute mostly
// padding: 127 experts of 4 rows (1536 x 2048) took it 47 us, of which the tensor core's work on whole tiles alone is
// 22 us, while the weights' bytes need 32. Persistent: two CTAs per SM walk the tiles (expert, 128 of its rows, 128
// weight rows) and the loads of the next tiles run ahead through the ring while a tile is finished. A tile of at
// most 32 rows loads 32 of the activation and takes them as its MMAs' columns, a larger one 128 and as many columns
// as it needs (a multiple of 32). Tiles start at multiples of 128 rows of their expert, so that their scales are
// whole blocks of the layout and start at the first column of their TMEM slot, as an MMA's scales have to.
constexpr int kGfRows = 128;
constexpr int kGfSmall = 32;
constexpr int kGfStages = 3;
// Taken for at most 32 rows per expert on average (all the host knows). 128 experts of 1536 x 2048, weights not in L2,
// this kernel against the pair kernel: 8 rows in all 8.6 / 10.1 us, 128 rows (80 experts) 28.2 / 31.7, 512 rows 37.0 /
// 46.9 (the weights' bytes need 31.5), 2048 rows 41.8 / 48.5, 4096 rows 44.0 / 49.3, 8192 rows 49.9 / 51.2.
// Other shapes at 32 and 64 rows per expert: 128 of 2048 x 768 25.9 / 30.2 and 34.6 / 33.0, 256 of 512 x 1024 20.8 / 23.2
// and 26.2 / 25.1, 8 of 4096 x 4096 17.7 / 21.2 and 19.1 / 21.8 (at 128 rows 27.6 / 22.9).
constexpr int64_t kGfMaxMeanRows = 32;

struct GfSmem {
    static constexpr int kA = 0;                                        // weight tiles
    static constexpr int kB = kA + kGfStages * 128 * 128;               // token tiles
    static constexpr int kSfa = kB + kGfStages * kGfRows * 128;
    static constexpr int kSfb = kSfa + kGfStages * kFewSf;
    static constexpr int kBar = kSfb + kGfStages * kFewSf;
    static constexpr int kMisc = kBar + (2 * kGfStages + 3) * 8;
    static constexpr int kGroups = (kMisc + 16 + 15) / 16 * 16;         // off, first 128-row tile
    static constexpr int kBytes = kGroups + 2 * (kMaxGroups + 1) * 4 + 1024;
};
static_assert(2 * (GfSmem::kBytes + 1024) <= 233472, "two CTAs per SM");

struct GfArgs {
    const int32_t* row_offsets;
    void* c;
    int64_t ldc;
    int M, N, K, G;
    int nkb, tiles_n;        // stages of 256 elements of K; 128-row tiles of a weight
    int out_bf16;
    uint32_t* err;
    uint64_t timeout_ns;
};

struct GfTile {
    int row0, rows;          // first row of A / C, rows of the tile
    int w_row0, w_tile;      // first weight row and scale tile (over all experts)
    int n0;                  // first column of C
    int sf_tile;             // A's scale tile
};

__device__ __forceinline__ GfTile gf_tile(const GfArgs& a, int t, const int32_t* off, const int32_t* pm128) {
    GfTile T;
    const int nt = t % a.tiles_n;
    T.sf_tile = t / a.tiles_n;
    const int g = find_group(pm128, a.G, T.sf_tile);
    T.row0 = off[g] + (T.sf_tile - pm128[g]) * kGfRows;
    T.rows = min(kGfRows, off[g + 1] - T.row0);
    T.n0 = nt * 128;
    T.w_row0 = g * a.N + T.n0;
    T.w_tile = g * a.tiles_n + nt;
    return T;
}

__global__ void __launch_bounds__(kFewThreads, 2)
    mx_grouped_gemm_fp4_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                                   const __grid_constant__ CUtensorMap tmap_x_small,
                                   const __grid_constant__ CUtensorMap tmap_sfw,
                                   const __grid_constant__ CUtensorMap tmap_sfx, const GfArgs a) {
    using L = GfSmem;
    constexpr int S = kGfStages;
    constexpr uint32_t kCols = 256, kSf = 128;  // TMEM: an accumulator of 128 columns, two scale slots of 8
    grid_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* empty = full + S;
    uint64_t* tmem_full = empty + S;
    uint64_t* acc_empty = tmem_full + 1;
    uint64_t* drain = acc_empty + 1;
    uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
    int32_t* off = reinterpret_cast<int32_t*>(smem + L::kGroups);
    int32_t* pm128 = off + (kMaxGroups + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(tmem_full, 1);
        mbar_init(acc_empty, 4);
        mbar_init(drain, 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmap_w);
        prefetch_tensormap(&tmap_x);
        prefetch_tensormap(&tmap_x_small);
        prefetch_tensormap(&tmap_sfw);
        prefetch_tensormap(&tmap_sfx);
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_slot, kCols);
        tmem_relinquish();
    }
    const int tiles = setup_groups<kGfRows>(a.row_offsets, a.G, a.M, a.err, off, pm128, nullptr, a.tiles_n);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_base_slot;

    if (warp == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const GfTile T = gf_tile(a, t, off, pm128);
            const bool small = T.rows <= kGfSmall;
            for (int kb = 0; kb < a.nkb; ++kb) {
                if (!mbar_wait_warp(&empty[stage], phase ^ 1u, abort, a.err, a.timeout_ns)) { ok = false; break; }
                mbar_arrive_expect_tx_elect(&full[stage],
                                            128 * 128 + (small ? kGfSmall : kGfRows) * 128 + 2 * kFewSf);
                tma_load_2d_elect(smem + L::kA + stage * 128 * 128, &tmap_w, &full[stage], kb * kBK, T.w_row0);
                if (small)
                    tma_load_2d_elect(smem + L::kB + stage * kGfRows * 128, &tmap_x_small, &full[stage], kb * kBK, T.row0);
                else
                    tma_load_2d_elect(smem + L::kB + stage * kGfRows * 128, &tmap_x, &full[stage], kb * kBK, T.row0);
                tma_load_3d_elect(smem + L::kSfa + stage * kFewSf, &tmap_sfw, &full[stage], 0, 4 * kb, T.w_tile);
                tma_load_3d_elect(smem + L::kSfb + stage * kFewSf, &tmap_sfx, &full[stage], 0, 4 * kb, T.sf_tile);
                if (issued < S) ++issued;
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
        // No copy may be in flight when the CTA leaves, whatever the other roles did.
        int s = stage;
        uint32_t p = phase;
        for (int i = 0; i < issued; ++i) {
            if (--s < 0) { s = S - 1; p ^= 1u; }
            mbar_wait_drain(&full[s], p, a.timeout_ns);
        }
    } else if (warp == 1) {
        int stage = 0, j = 0;
        uint32_t phase = 0, empty_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++j) {
            const GfTile T = gf_tile(a, t, off, pm128);
            if (j > 0) {                        // the previous tile has been read out of the accumulator
                if (!mbar_wait_warp(acc_empty, empty_phase, abort, a.err, a.timeout_ns)) break;
                empty_phase ^= 1u;
            }
            tc_fence_after();
            const uint32_t cols = static_cast<uint32_t>((T.rows + 31) / 32 * 32);
            const uint32_t idesc[2] = {idesc_mxf4(128, cols, 0), idesc_mxf4(128, cols, 2)};
            for (int kb = 0; kb < a.nkb; ++kb) {
                if (!mbar_wait_warp(&full[stage], phase, abort, a.err, a.timeout_ns)) { ok = false; break; }
                tc_fence_after();
                const uint64_t adesc = sdesc_kmajor_sw128(smem_u32(smem + L::kA + stage * 128 * 128));
                const uint64_t bdesc = sdesc_kmajor_sw128(smem_u32(smem + L::kB + stage * kGfRows * 128));
                const uint64_t sda = sdesc_scale_block(smem_u32(smem + L::kSfa + stage * kFewSf));
                const uint64_t sdb = sdesc_scale_block(smem_u32(smem + L::kSfb + stage * kFewSf));
                const int left = a.K - kb * 256;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tc_cp_elect(tmem_base + kSf + 8u * h, sda + 32u * h);
                    tc_cp_elect(tmem_base + kSf + 8u * h + 4u, sdb + 32u * h);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t id = 2u * (k & 1), sfa_t = tmem_base + kSf + 8u * (k >> 1);
                    if (64 * k < left)
                        tc_mma_mxf4_elect(tmem_base, adesc + 2u * k, bdesc + 2u * k, idesc[k & 1], sfa_t | (id << 30),
                                          (sfa_t + 4u) | (id << 30), (kb | k) != 0 ? 1u : 0u);
                }
                tc_commit_elect(&empty[stage]);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            tc_commit_elect(tmem_full);
        }
        // Every MMA issued by this warp has completed once `drain` fires.
        __syncwarp();
        tc_commit_elect(drain);
        mbar_wait_drain(drain, 0, a.timeout_ns);
    } else {
        // Lane l of quadrant q is weight row 32 q + l, accumulator column m row m of the tile.
        const int q = warp & 3;
        uint32_t full_phase = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const GfTile T = gf_tile(a, t, off, pm128);
            if (!mbar_wait_warp(tmem_full, full_phase, abort, a.err, a.timeout_ns)) break;
            full_phase ^= 1u;
            tc_fence_after();
            const int n = T.n0 + 32 * q + lane;
            for (int m0 = 0; m0 < T.rows; m0 += 32) {
                uint32_t r[32];
                tc_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + m0, r);
                tc_wait_ld_regs(r);
                if (m0 + 32 >= T.rows) {        // the last of the tile is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty);
                }
                const int64_t at = static_cast<int64_t>(T.row0 + m0) * a.ldc + n;
                if (n < a.N) {
                    if (a.out_bf16) {
                        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(a.c) + at;
#pragma unroll
                        for (int m = 0; m < 32; ++m)
                            if (m0 + m < T.rows) c[m * a.ldc] = __float2bfloat16_rn(__uint_as_float(r[m]));
                    } else {
                        float* c = static_cast<float*>(a.c) + at;
#pragma unroll
                        for (int m = 0; m < 32; ++m)
                            if (m0 + m < T.rows) c[m * a.ldc] = __uint_as_float(r[m]);
                    }
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kCols);
    }
}

}  // namespace mx
