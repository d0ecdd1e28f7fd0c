// Attention over the paged E4M3 cache (cache.cuh) for few rows per sequence: decoding steps.
//
//   out[r] = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale q_r . k_j),   j the keys that row r sees
//
// Bound by one pass over the visible codes. G = Hq / Hkv query heads share a key head; their rows (and those of a sequence's
// few new tokens) are one tile, so that the codes are read once. Products are transposed: S^T = K q^T and O^T = V^T P^T
// with 16 tokens (or 16 features) as the rows of mma.m16n8k16 and 8 query rows as its columns, which wastes no lane at 8 rows.
// mma.sync and not tcgen05: at G rows the tensor work is 1 / 16 of what the bytes allow, and operands go from the ring
// of codes to registers by conversion (E4M3 -> f16 is exact, one instruction for two), where tcgen05 would want them
// written back to shared memory.
//
// Types: q rows are scaled by a power of two each and become f16 (exact but for elements 2^29 below the row's largest); S, softmax
// statistics and O are fp32. A page's key scale enters with the softmax's argument t, its value scale with P's exponent: P =
// 2^(t + e - M + 7), e the exponent of the page's values and M a whole number near the largest t + e that the row sees, so that
// P, as f16, has 11 bits from 2^-20 of the row's largest product of weight and value scale up, however far scales lie apart and
// whatever pages it does not see hold. The sum l of the weights has a reference of its own, the largest t, kept as the distance
// `lift` of M from it: l takes P 2^(lift - e - 7) from P in fp32, and where e lies so far below M's that P would leave fp32's
// range, both take e to be lift - 100 (2^-93 of the row's largest: 0 as f16 in either case). M and lift are moved only when P would
// leave f16's range (8 binades) or l grows by 2^40, so that O is seldom rescaled.
//
// Work is split evenly: every sequence, key head and tile of rows has its keys cut into steps of 64, and block i of n takes the
// i-th n-th of all steps, wherever it begins and ends. Blocks that share a tile leave (O, M, l) in a workspace, which
// a second kernel joins; sums are made in the order of the keys. Each of a block's four warps streams its own 16 tokens of
// a step through a private ring of cp.async stages: no block-wide wait until a tile ends.
//
// 64 tokens over 2000 to 8000 keys of 8 heads of 128 (628 MB): 113 us, 106 of them here (5.9 TB/s); 4 over 30 000 to 120 000 of 4 heads
// (381 MB): 83 us, 73 of them here; one over 1000: 10.5 us, nearly all of it chains of loads.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "cache.cuh"
#include "ptx.cuh"

namespace mx {

constexpr int kAtThreads = 128;
constexpr int kAtWarps = kAtThreads / 32;
constexpr int kAtStep = 64;            // keys per step: 16 per warp
constexpr float kAtBias = 7.0f;        // P = 2^(t + e - M + 7)
constexpr float kAtSlack = 8.0f;       // M lags behind the maximum by at most this
constexpr float kAtSumSlack = 40.0f;   // weights in l reach at most 2^40
constexpr float kAtNone = -1e30f;      // M of a row that has seen no key
constexpr float kAtLeast = 100.0f;     // exponents of value scales below lift - 100 count as that

struct AttendArgs {
    CacheView c;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;                   // [T, Hq], or null
    float* parts;                 // workspace
    int64_t ldq_t, ldq_h, ldo_t, ldo_h;
    int64_t window;               // keys a row sees; 2^62: all
    float scale_log2;
    uint32_t* err;
    uint64_t timeout_ns;
    int Hq, G;
    FastDiv group;                // G
    int blocks;                   // blocks that share the steps
    int most_rows;                // sequences with more rows (new tokens x G) are left to the kernel for many
    int min_steps;                // steps that a block takes at least
    uint8_t* plan;                // of the kernel for many rows, written by this one's last block; null: no such sequences
    float* many_parts;
    int many_blocks, plan_items;  // its blocks; items that the plan has room for
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(x - 127) of a whole number x <= 254; 0 below 1.
__device__ __forceinline__ float pow2_biased(float x) {
    return __int_as_float(__float_as_int(fmaxf(x, 0.0f) + 8388608.0f) << 23);      // the sum's last bits are x
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void copy16(uint32_t saddr, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr), "l"(g) : "memory");
}
// 16 bytes to shared memory; zeros where `have` is 0.
__device__ __forceinline__ void copy16(uint32_t saddr, const void* g, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(saddr), "l"(g), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- what there is to do -------------------------------------------------------------------------------------

// A sequence as the kernel for few rows sees it: `rows` query rows per key head, keys [lo, hi) seen by some of them, cut
// into `steps` steps from lo rounded down, each of `tiles` tiles of rows. No rows, or more than most_rows: nothing to do.
struct Sequence {
    int first, n, rows, tiles;
    int64_t lo, hi, steps;
};
template <int ROWS>
__device__ __forceinline__ Sequence sequence(const AttendArgs& a, int b) {
    Sequence s;
    rows_of(a.c, b, s.first, s.n);
    s.rows = s.n * a.G;
    if (s.rows > a.most_rows) s.rows = 0;
    s.tiles = (s.rows + ROWS - 1) / ROWS;
    s.hi = max(a.c.lengths[b], 0);
    s.lo = max(s.hi - s.n - a.window + 1, int64_t(0)) & ~int64_t(kAtStep - 1);
    if (s.lo > s.hi) s.lo = s.hi;
    s.steps = max((s.hi - s.lo + kAtStep - 1) / kAtStep, int64_t(1));      // a row without keys is written too
    return s;
}

// Steps of all sequences before `b` and of all of them, by a whole block: thread t sums a stretch of consecutive sequences.
// `find` >= 0: the sequence that holds step `find` instead (its number in `b`).
template <int ROWS, int THREADS>
struct Steps {
    int64_t sums[THREADS];       // of the threads' stretches, then their prefix
    int64_t total, before;
    int found;
};
template <int ROWS, int THREADS>
__device__ __forceinline__ void count_steps(const AttendArgs& a, Steps<ROWS, THREADS>& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.c.B + THREADS - 1) / THREADS;
    int64_t sum = 0;
    for (int b = tid * per; b < min((tid + 1) * per, a.c.B); ++b) {
        const Sequence q = sequence<ROWS>(a, b);
        sum += q.steps * q.tiles * a.c.Hkv;
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
    }
    __shared__ int64_t warps[THREADS / 32];
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    int64_t at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warps[w];
    s.sums[tid] = at;
    if (tid == THREADS - 1) s.total = at + sum;
    __syncthreads();
}
// After count_steps: the steps before sequence b.
template <int ROWS, int THREADS>
__device__ __forceinline__ int64_t steps_before(const AttendArgs& a, const Steps<ROWS, THREADS>& s, int b) {
    const int per = (a.c.B + THREADS - 1) / THREADS, t = b / per;
    int64_t at = s.sums[t];
    for (int i = t * per; i < b; ++i) {
        const Sequence q = sequence<ROWS>(a, i);
        at += q.steps * q.tiles * a.c.Hkv;
    }
    return at;
}
// After count_steps, by the whole block: the sequence that holds step x (x < total) and the steps before it.
template <int ROWS, int THREADS>
__device__ __forceinline__ void find_step(const AttendArgs& a, Steps<ROWS, THREADS>& s, int64_t x) {
    const int tid = threadIdx.x;
    const int per = (a.c.B + THREADS - 1) / THREADS;
    const int64_t end = tid + 1 < THREADS ? s.sums[tid + 1] : s.total;
    if (s.sums[tid] <= x && x < end) {
        int64_t at = s.sums[tid];
        for (int b = tid * per; b < min((tid + 1) * per, a.c.B); ++b) {
            const Sequence q = sequence<ROWS>(a, b);
            const int64_t n = q.steps * q.tiles * a.c.Hkv;
            if (x < at + n) {
                s.found = b;
                s.before = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ int64_t share_of(const AttendArgs& a, int64_t total) {
    return max((total + a.blocks - 1) / a.blocks, int64_t(a.min_steps));
}

// What a quotient O / l is in units of, for M - lift = M's distance from the reference of l. (An exponent that P's own cannot have
// stands for rows of infinities, whose quotients are NaN.)
__device__ __forceinline__ float out_unit(float lift) { return ldexpf(1.0f, static_cast<int>(fminf(fmaxf(lift - kAtBias, -300.0f), 300.0f))); }

// Floats of one part: O [ROWS][D], then M, l and lift [ROWS] each.
__host__ __device__ constexpr int64_t part_floats(int rows, int D) { return int64_t(rows) * (D + 3); }

// ---- the plan of the kernel for many rows (attend_many.cuh) ------------------------------------------------------
// Sequences with more rows than most_rows are cut into items of 256 rows. An item of every key head is a unit of work of as many
// key tiles (128) as its rows see. The cost of all units, item by item and head by head, is shared evenly among the blocks: a
// unit costs its tiles, and kAmUnitCost in front of them for what is done once per unit. The plan lists the items and the cost
// in front of each.

constexpr int kAmRows = 256;           // query rows of an item
constexpr int kAmKeys = 128;           // keys per tile
constexpr int kAmUnitCost = 3;         // in tiles: 15 000 cycles of queries, output and a first tile's start, 4600 a tile (heads of 128; taken for 64 too)

struct alignas(16) AmItem {
    int64_t at;                        // cost of all units in front of the item
    int32_t b, row0, rows;             // sequence; its query rows [row0, row0 + rows)
    int32_t first, n, hi;              // the sequence's rows in the batch, its keys
    int32_t lo;                        // first key of the item's tiles (a multiple of 16)
    int32_t tiles[2];                  // key tiles of the first 128 rows and of the others
    int32_t unused;
};
constexpr int kAmMaxBlocks = 160;      // of the kernel for many rows
struct alignas(16) AmHeader {
    int64_t total;                     // cost of all units
    int32_t items, unused;
    int32_t done[kAmMaxBlocks];        // blocks whose parts are complete (no wait of theirs has run out)
};
__device__ __forceinline__ AmHeader* plan_header(const AttendArgs& a) { return reinterpret_cast<AmHeader*>(a.plan); }
__device__ __forceinline__ AmItem* plan_item(const AttendArgs& a, int i) { return reinterpret_cast<AmItem*>(a.plan + sizeof(AmHeader)) + i; }
// Tiles of a unit; one at least, since rows without keys are written too.
__device__ __forceinline__ int unit_tiles(const AmItem& w) { return max(max(w.tiles[0], w.tiles[1]), 1); }
__device__ __forceinline__ int64_t unit_cost(const AmItem& w) { return unit_tiles(w) + kAmUnitCost; }

__device__ __forceinline__ void set_rows(const AttendArgs& a, AmItem& w, int64_t row0) {
    w.row0 = static_cast<int>(row0);
    w.rows = static_cast<int>(min(int64_t(w.n) * a.G - row0, int64_t(kAmRows)));
    const int64_t start = int64_t(w.hi) - w.n;                   // position of the sequence's first row
    w.lo = static_cast<int>(min(max(start + a.group.div(w.row0) - a.window + 1, int64_t(0)), int64_t(w.hi)) & ~int64_t(15));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int end = min(w.rows, (t + 1) * 128);              // rows of the halves 0 .. t
        const int64_t last = end > t * 128 ? start + a.group.div(w.row0 + end - 1) : -1;
        w.tiles[t] = last < w.lo ? 0 : static_cast<int>((last - w.lo) / kAmKeys) + 1;
    }
}

// By one block: thread t lists the items of a stretch of consecutive sequences.
template <int THREADS>
__device__ __forceinline__ void write_plan(const AttendArgs& a) {
    __shared__ int64_t warps[2][THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.c.B + THREADS - 1) / THREADS;
    for (int i = tid; i < kAmMaxBlocks; i += THREADS) plan_header(a)->done[i] = 0;
    int64_t items = 0, cost = 0;
    auto walk = [&](bool write, int64_t at, int64_t before) {
        AmItem w;
        for (int b = tid * per; b < min((tid + 1) * per, a.c.B); ++b) {
            rows_of(a.c, b, w.first, w.n);
            const int64_t rows = int64_t(w.n) * a.G;
            if (rows <= a.most_rows) continue;
            w.b = b;
            w.hi = max(a.c.lengths[b], 0);
            for (int64_t row0 = 0; row0 < rows; row0 += kAmRows) {
                set_rows(a, w, row0);
                w.at = before;
                if (write && at < a.plan_items) *plan_item(a, static_cast<int>(at)) = w;
                ++at;
                before += unit_cost(w) * a.c.Hkv;
            }
        }
        items = at;
        cost = before;
    };
    walk(false, 0, 0);
    int64_t si = items, st = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ui = __shfl_up_sync(0xFFFFFFFFu, si, o), ut = __shfl_up_sync(0xFFFFFFFFu, st, o);
        if (lane >= o) si += ui, st += ut;
    }
    if (lane == 31) warps[0][warp] = si, warps[1][warp] = st;
    __syncthreads();
    si -= items, st -= cost;
    for (int w = 0; w < warp; ++w) si += warps[0][w], st += warps[1][w];
    walk(true, si, st);
    if (tid == THREADS - 1) {
        // More items than the batch's rows can make: offsets that name rows twice. Nothing is computed then.
        const bool good = items <= a.plan_items;
        plan_header(a)->total = good ? cost : 0;
        plan_header(a)->items = good ? static_cast<int32_t>(items) : 0;
        if (!good) atomicOr(a.err, kErrBadOffsets);
    }
}

template <int D, int NT>
struct AtSmem {
    static constexpr int kStage = 2 * 16 * D;                     // keys, then values
    static constexpr int kBlocks = NT == 1 ? 3 : 2;               // an SM's
    static constexpr int kStages = (NT == 1 ? 4 : 6) * 128 / D;
    static constexpr int kWarp = kStages * kStage;                // a warp's ring; at the end of a tile, its O
    static constexpr int kBytes = kAtWarps * kWarp;
    static_assert(8 * NT * (D + 4) * 4 <= kWarp, "a warp's O takes the place of its ring");
};

// The 16-byte pieces of a row are stored in an order that depends on the row, so that both the keys' reads (eight lanes: two
// rows, four pieces) and the values' (four rows 2c, two pieces) meet every bank once.
template <int D>
__device__ __forceinline__ int ring_piece(int row, int piece) {
    return D == 128 ? piece ^ ((row & 6) ^ ((row & 1) << 2)) : piece ^ ((row >> 1) & 3);
}

template <int D, int NT>
__global__ void __launch_bounds__(kAtThreads, NT == 1 ? 3 : 2) attend_few_kernel(const __grid_constant__ AttendArgs a) {
    grid_wait();
    constexpr int ROWS = 8 * NT;
    using S = AtSmem<D, NT>;
    constexpr int kS = S::kStages;
    constexpr int KS = D / 16;                  // k-steps of S^T, and tiles of 16 features of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Steps<ROWS, kAtThreads> todo;
    __shared__ float stat[kAtWarps][3][ROWS];
    const CacheView& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
    if (static_cast<int>(blockIdx.x) == a.blocks) {          // there is such a block where a.plan is set
        write_plan<kAtThreads>(a);
        return;
    }
    count_steps<ROWS, kAtThreads>(a, todo);
    const int64_t share = share_of(a, todo.total);
    int64_t at = blockIdx.x * share;
    const int64_t stop = min(at + share, todo.total);
    if (at >= stop) return;
    find_step<ROWS, kAtThreads>(a, todo, at);
    int b = todo.found;
    int64_t before = todo.before;
    const uint32_t ring = smem_u32(smem) + warp * S::kWarp;
    const uint8_t* ring_p = smem + warp * S::kWarp;
    Sequence sq = sequence<ROWS>(a, b);

    while (at < stop) {
        while (at >= before + sq.steps * sq.tiles * c.Hkv) {           // on to the sequence that holds `at`
            before += sq.steps * sq.tiles * c.Hkv;
            sq = sequence<ROWS>(a, ++b);
        }
        const int64_t in_seq = at - before, unit = in_seq / sq.steps;
        const int64_t s0 = in_seq - unit * sq.steps, s1 = min(sq.steps, s0 + (stop - at));
        const int h = static_cast<int>(unit / sq.tiles), tile = static_cast<int>(unit - int64_t(h) * sq.tiles);
        const int row0 = tile * ROWS;

        float o[NT][KS][4], M[NT][2], l[NT][2], lift[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < KS; ++k) o[nt][k][0] = o[nt][k][1] = o[nt][k][2] = o[nt][k][3] = 0.0f;
            M[nt][0] = M[nt][1] = kAtNone;
            l[nt][0] = l[nt][1] = lift[nt][0] = lift[nt][1] = 0.0f;
        }

        // Pages of 32 steps, a lane each, one batch ahead: (page id, scale bytes).
        const int steps = static_cast<int>(s1 - s0);
        const int64_t tok0 = sq.lo + s0 * kAtStep + 16 * warp;
        const int key0 = static_cast<int>(s0 * kAtStep) + 16 * warp;
        int64_t next_id = -1, cur_id = -1;
        uint32_t next_sc = 0xFFFF, cur_sc = 0xFFFF, last_sc = 0xFFFF;
        auto fetch_ids = [&](int base) {
            const int64_t tok = tok0 + int64_t(base + lane) * kAtStep;
            next_id = -1;
            // 16 keys in front of the first row's window, whose page may be another sequence's by now, are as if behind the end: masked.
            if (base + lane < steps && tok < sq.hi && tok + 16 > sq.hi - sq.n - a.window + 1) {
                next_id = page_id(c, b, tok >> c.page_shift);
                if (next_id < 0) atomicOr(a.err, kErrBadIndex);
            }
        };
        auto fetch_scales = [&]() {
            next_sc = 0xFFFFu;
            if (next_id >= 0) next_sc = c.ks[next_id * c.ks_page + h] | static_cast<uint32_t>(c.vs[next_id * c.vs_page + h]) << 8;
        };
        // Where the lane's pieces of a step go, piece i at to[i % 2] + 512 i: the order of a row's pieces repeats every 8 rows.
        uint32_t to[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (i * 32 + lane) / (D / 16), piece = lane % (D / 16);
            to[i] = row * D + ring_piece<D>(row, piece) * 16 - i * 512;
        }
        int put = 0;                            // steps whose copies are issued
        auto issue = [&]() {
            if (put < steps) {
                const int in = put & 31;
                if (in == 0) {
                    if (put == 0) {
                        fetch_ids(0);
                        fetch_scales();                // looked at with the first scores
                    }
                    cur_id = next_id;
                    last_sc = cur_sc;
                    cur_sc = next_sc;
                    fetch_ids(put + 32);
                }
                if (in == 16) fetch_scales();
                const int64_t id = __shfl_sync(0xFFFFFFFFu, cur_id, in);
                const int stage = put % kS;
                const int64_t tok = tok0 + int64_t(put) * kAtStep;
                const int64_t inner = ((static_cast<int64_t>(h) << c.page_shift) + (tok & ((1 << c.page_shift) - 1))) * D + lane * 16;
                const uint8_t* kp = c.k + (id * c.k_page + inner);
                const uint8_t* vp = c.v + (id * c.v_page + inner);
                const uint32_t dst = ring + stage * S::kStage;
                if (id >= 0 && tok + 16 <= sq.hi) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        copy16(dst + to[i % 2] + i * 512, kp + i * 512);
                        copy16(dst + to[i % 2] + i * 512 + 16 * D, vp + i * 512);
                    }
                } else {
                    __syncwarp();
                    const int valid = id < 0 ? 0 : static_cast<int>(max(min(sq.hi - tok, int64_t(16)), int64_t(0)));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const bool have = (i * 32 + lane) / (D / 16) < valid;
                        copy16(dst + to[i % 2] + i * 512, have ? static_cast<const void*>(kp + i * 512) : a.q, have);
                        copy16(dst + to[i % 2] + i * 512 + 16 * D, have ? static_cast<const void*>(vp + i * 512) : a.q, have);
                    }
                }
                ++put;
            }
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < kS - 1; ++i) issue();

        // The first keys are on their way.
        // Queries: column n = 8 nt + g of S^T is row row0 + n. Lane (g, c4) holds the features of the pieces that
        // lane (., c4) holds of a key: pieces c4 and c4 + 4 (D = 128), or c4 (D = 64).
        uint32_t qf[NT][KS][2];
        float rowf[NT][2];                      // argument of 2^x per unit of S, of columns 2 c4 and 2 c4 + 1
        int stop[NT][2], start[NT][2];          // keys that these columns see, [start, stop), counted from sq.lo
        int all_from = 0, all_to = INT_MAX;     // keys that every column of the tile that has a row sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + 8 * nt + g;
            const bool have = r < sq.rows;
            const int tok = have ? a.group.div(r) : 0;
            const __nv_bfloat16* src = a.q + (sq.first + tok) * a.ldq_t + (h * a.G + (r - tok * a.G)) * a.ldq_h;
            float x[D / 4];
            uint32_t m = 0;
#pragma unroll
            for (int p = 0; p < D / 64; ++p)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 w = have ? *reinterpret_cast<const uint4*>(src + (c4 + 4 * p) * 16 + i * 8) : make_uint4(0, 0, 0, 0);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[p * 16 + i * 8 + 2 * j] = bf16_lo(u[j]);
                        x[p * 16 + i * 8 + 2 * j + 1] = bf16_hi(u[j]);
                        m = max(m, max(u[j] & 0x7FFFu, (u[j] >> 16) & 0x7FFFu));
                    }
                }
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            // 2^(141 - E): the largest element lands in [2^14, 2^15). A row with NaN or infinity, or of zeros, stays as it is.
            const int E = static_cast<int>(m >> 7);
            const int up = E == 255 || m == 0 ? 0 : min(max(141 - E, -126), 126);
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23), div = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[nt][k][0] = f16x2(x[4 * k] * mul, x[4 * k + 1] * mul);
                qf[nt][k][1] = f16x2(x[4 * k + 2] * mul, x[4 * k + 3] * mul);
            }
            const float f = a.scale_log2 * div;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                rowf[nt][j] = __shfl_sync(0xFFFFFFFFu, f, (2 * c4 + j) * 4);
                const int col = row0 + 8 * nt + 2 * c4 + j;
                const int64_t last = col < sq.rows ? sq.hi - sq.n + a.group.div(col) : -1;
                stop[nt][j] = static_cast<int>(max(last + 1 - sq.lo, int64_t(0)));
                start[nt][j] = static_cast<int>(max(last - a.window + 1 - sq.lo, int64_t(0)));
                if (col < sq.rows) {
                    all_from = max(all_from, start[nt][j]);
                    all_to = min(all_to, stop[nt][j]);
                }
            }
        }

        all_from = __reduce_max_sync(0xFFFFFFFFu, all_from);
        all_to = __reduce_min_sync(0xFFFFFFFFu, all_to);
        for (int st = 0; st < steps; ++st) {
            copies_wait<kS - 2>();
            __syncwarp();
            issue();                             // into the stage that the last step left
            const int stage = st % kS;
            const uint8_t* kr = ring_p + stage * S::kStage;
            const uint8_t* vr = kr + 16 * D;
            // Its scales: of the batch that copies are issued from, or of the one before it.
            const uint32_t sc = __shfl_sync(0xFFFFFFFFu, st >> 5 == (put - 1) >> 5 ? cur_sc : last_sc, st & 31);
            const int key = key0 + st * kAtStep;       // the first of the 16, from sq.lo

            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
            for (int p = 0; p < D / 64; ++p) {
                const uint4 x = *reinterpret_cast<const uint4*>(kr + g * D + ring_piece<D>(g, c4 + 4 * p) * 16);
                const uint4 y = *reinterpret_cast<const uint4*>(kr + (g + 8) * D + ring_piece<D>(g + 8, c4 + 4 * p) * 16);
                const uint32_t xu[4] = {x.x, x.y, x.z, x.w}, yu[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t a0 = f16x2_of_e4m3(xu[w]), a1 = f16x2_of_e4m3(yu[w]);
                    const uint32_t a2 = f16x2_of_e4m3_hi(xu[w]), a3 = f16x2_of_e4m3_hi(yu[w]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a0, a1, a2, a3, qf[nt][4 * p + w][0], qf[nt][4 * p + w][1]);
                }
            }
            // 2^x arguments of (token g, columns 2 c4, 2 c4 + 1), (token g + 8, the same columns).
            const uint32_t kb = sc & 0xFFu, vb = sc >> 8;
            const float kscale = kb == 255 ? __uint_as_float(0x7FC00000u) : scale_value(kb);
            const float e = vb == 255 ? 0.0f : static_cast<float>(static_cast<int>(vb) - 127);
            bool more = false;
            const bool edge = key < all_from || key > all_to - 16;       // key + 16 may pass 2^31 - 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f0 = rowf[nt][0] * kscale, f1 = rowf[nt][1] * kscale;
                s[nt][0] *= f0, s[nt][1] *= f1, s[nt][2] *= f0, s[nt][3] *= f1;
            }
            if (edge) {
                __syncwarp();                          // a branch and not selections in every step
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = key + g + 8 * (i >> 1);
                        if (at >= stop[nt][i & 1] || at < start[nt][i & 1]) s[nt][i] = -INFINITY;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    more |= fmaxf(s[nt][j], s[nt][2 + j]) > M[nt][j] + fminf(kAtSlack - e, kAtSumSlack - lift[nt][j]);
            if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float m = fmaxf(s[nt][j], s[nt][2 + j]);
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                        const float to = fmaxf(M[nt][j], rintf(m + e)), f = exp2_approx(M[nt][j] - to);
                        const float up = to - fmaxf(M[nt][j] - lift[nt][j], rintf(m));
                        l[nt][j] *= exp2_approx((M[nt][j] - to) - (lift[nt][j] - up));
                        M[nt][j] = to;
                        lift[nt][j] = up;
#pragma unroll
                        for (int k = 0; k < KS; ++k) o[nt][k][j] *= f, o[nt][k][2 + j] *= f;
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float el = fmaxf(e, lift[nt][j] - kAtLeast), d = el - (M[nt][j] - kAtBias);
                    p[j] = exp2_approx(s[nt][j] + d);                   // 0 of -inf: M is finite
                    p[2 + j] = exp2_approx(s[nt][2 + j] + d);
                    l[nt][j] += (p[j] + p[2 + j]) * pow2_biased(lift[nt][j] + (127.0f - kAtBias) - el);
                }
                if (vb == 255)                                          // values that are NaN
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = s[nt][i] != -INFINITY ? __uint_as_float(0x7FC00000u) : 0.0f;
                pf[nt][0] = transposed8x8(f16x2(p[0], p[1]));
                pf[nt][1] = transposed8x8(f16x2(p[2], p[3]));
            }
            // Lane (g, c4): features D / 8 g .. of tokens 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9. Rows g and g + 8 of
            // feature tile k are features D / 8 g + 2 k and + 2 k + 1.
            uint32_t vw[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * c4 + (i & 1) + 8 * (i >> 1);
                if constexpr (D == 128) {
                    const uint4 w = *reinterpret_cast<const uint4*>(vr + row * D + ring_piece<D>(row, g) * 16);
                    vw[i][0] = w.x, vw[i][1] = w.y, vw[i][2] = w.z, vw[i][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(vr + row * D + ring_piece<D>(row, g >> 1) * 16 + (g & 1) * 8);
                    vw[i][0] = w.x, vw[i][1] = w.y;
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), x1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                const uint32_t y0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), y1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t x = k ? x1 : x0, y = k ? y1 : y0;
                    const uint32_t a0 = f16x2_of_e4m3(x), a1 = f16x2_of_e4m3_hi(x), a2 = f16x2_of_e4m3(y), a3 = f16x2_of_e4m3_hi(y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * w + k], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            }
        }

        // The four warps' parts, joined in shared memory: M, l and lift per row, O relative to the largest M, l to the largest
        // M - lift. No copy is in flight: the last groups are empty.
        copies_wait<0>();
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = l[nt][j];
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
                const int n = 8 * nt + 2 * c4 + j;
                if (g == 0) {
                    stat[warp][0][n] = M[nt][j];
                    stat[warp][1][n] = x;
                    stat[warp][2][n] = lift[nt][j];
                }
                float* dst = reinterpret_cast<float*>(smem + warp * S::kWarp) + n * (D + 4) + g * (D / 8);
#pragma unroll
                for (int k = 0; k < KS; ++k) *reinterpret_cast<float2*>(dst + 2 * k) = make_float2(o[nt][k][j], o[nt][k][2 + j]);
            }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == sq.steps;
        float* part = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (s0 == 0 ? 1 : 0)) * part_floats(ROWS, D);
        for (int n = warp; n < ROWS && row0 + n < sq.rows; n += kAtWarps) {
            float top = kAtNone, ref = kAtNone, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) {
                top = fmaxf(top, stat[w][0][n]);
                ref = fmaxf(ref, stat[w][0][n] - stat[w][2][n]);
            }
            float acc[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) {
                const float lw = stat[w][1][n];
                if (lw == 0.0f) continue;        // no key seen: nothing of this warp counts
                const float f = exp2_approx(stat[w][0][n] - top);
                sum += lw * exp2_approx(stat[w][0][n] - stat[w][2][n] - ref);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) acc[i] += f * reinterpret_cast<const float*>(smem + w * S::kWarp)[n * (D + 4) + lane + 32 * i];
            }
            if (whole) {
                const int r = row0 + n, tok = a.group.div(r), head = h * a.G + (r - tok * a.G);
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, unit = out_unit(top - ref);
                __nv_bfloat16* dst = a.out + (sq.first + tok) * a.ldo_t + head * a.ldo_h;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) dst[lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv * unit);
                if (a.lse && lane == 0)
                    a.lse[static_cast<int64_t>(sq.first + tok) * a.Hq + head] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.693147180559945f;
            } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) part[n * D + lane + 32 * i] = acc[i];
                if (lane == 0) {
                    part[ROWS * D + n] = top;
                    part[ROWS * D + ROWS + n] = sum;
                    part[ROWS * D + 2 * ROWS + n] = top - ref;
                }
            }
        }
        __syncthreads();
        at += s1 - s0;
    }
}

constexpr int kAtJoinThreads = 256;

// Joins the parts of tiles whose steps went to several blocks: a block per (sequence, key head, tile of rows), a warp per
// row. Parts are added in the order of their keys.
template <int D, int NT>
__device__ __forceinline__ void join_few(const AttendArgs& a, int tiles) {
    constexpr int ROWS = 8 * NT;
    __shared__ Steps<ROWS, kAtJoinThreads> todo;
    const CacheView& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % c.Hkv, b = blockIdx.x / tiles / c.Hkv;
    const Sequence sq = sequence<ROWS>(a, b);
    if (tile >= sq.tiles) return;
    count_steps<ROWS, kAtJoinThreads>(a, todo);
    const int64_t share = share_of(a, todo.total);
    const int64_t s0 = steps_before<ROWS, kAtJoinThreads>(a, todo, b) + (int64_t(h) * sq.tiles + tile) * sq.steps;
    const int64_t i0 = s0 / share, i1 = (s0 + sq.steps - 1) / share;
    if (i0 == i1) return;
    const int parts = static_cast<int>(i1 - i0) + 1;
    // Part 0 is the second of its block's two, the others the first of theirs.
    auto part = [&](int i) { return a.parts + (2 * (i0 + i) + (i == 0 ? 1 : 0)) * part_floats(ROWS, D); };
    constexpr int W = D / 32;                        // features of a lane
    for (int n = warp; n < ROWS && tile * ROWS + n < sq.rows; n += kAtJoinThreads / 32) {
        float acc[W], sum = 0.0f, top = kAtNone, ref = kAtNone;
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = 0.0f;
        for (int i = 0; i < parts; i += 16) {
            // 16 parts at a time: O, and M, l and lift (lane l those of part i + l), all on their way at once.
            float v[16][W];
            const bool have = lane < 16 && i + lane < parts;
            const float* mine = part(i + (have ? lane : 0)) + ROWS * D + n;
            const float M = have ? mine[0] : kAtNone, ls = have ? mine[ROWS] : 0.0f, L = M - (have ? mine[2 * ROWS] : 0.0f);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float* p = part(min(i + k, parts - 1)) + n * D + lane * W;
                if constexpr (W == 4)
                    *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(p);
                else
                    *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(p);
            }
            float next = fmaxf(top, M), base = fmaxf(ref, L);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                next = fmaxf(next, __shfl_xor_sync(0xFFFFFFFFu, next, o));
                base = fmaxf(base, __shfl_xor_sync(0xFFFFFFFFu, base, o));
            }
            next = __shfl_sync(0xFFFFFFFFu, next, 0);
            base = __shfl_sync(0xFFFFFFFFu, base, 0);
            const float back = exp2_approx(top - next), f = have ? exp2_approx(M - next) : 0.0f;
            const float weight = have ? ls * exp2_approx(L - base) : 0.0f;
            sum *= exp2_approx(ref - base);
            top = next;
            ref = base;
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] *= back;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (i + k >= parts) break;
                const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
                sum += __shfl_sync(0xFFFFFFFFu, weight, k);
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j] += fk * v[k][j];
            }
        }
        const int r = tile * ROWS + n, tok = a.group.div(r), head = h * a.G + (r - tok * a.G);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, unit = out_unit(top - ref);
        __nv_bfloat16* dst = a.out + (sq.first + tok) * a.ldo_t + head * a.ldo_h + lane * (D / 32);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) dst[j] = __float2bfloat16_rn(acc[j] * inv * unit);
        if (a.lse && lane == 0)
            a.lse[static_cast<int64_t>(sq.first + tok) * a.Hq + head] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.693147180559945f;
    }
}

}  // namespace mx
