// Inline-PTX helpers for sm_100a: mbarriers, TMA / bulk copies (none with multicast), tcgen05
// (TMEM, UMMA), timers.
// Everything here is a one-instruction wrapper; no arithmetic of the method lives in this file.
#pragma once
#include <cstdint>
#include <cuda.h>

namespace mx {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// ---- mbarrier -------------------------------------------------------------------------------

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Error bits recorded in the device status word.
enum : uint32_t {
    kErrWaitTimeout = 1u,      // an mbarrier wait ran past its deadline
    kErrBadOffsets = 2u,       // grouped GEMM: row offsets not 0 .. total_rows, nondecreasing
};

// Bounded wait: returns true once the phase with `parity` has completed; false if `abort` was
// raised by another role, or if `timeout_ns` passed (then it raises `abort` and sets `err`).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* err, uint64_t timeout_ns) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(a, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > timeout_ns) {
            *abort = 1;
            atomicOr(err, kErrWaitTimeout);
            return false;
        }
    }
}

// mbar_wait by a whole warp with one answer for all its lanes. Every role that goes on to a warp-wide instruction
// (elect.sync, tcgen05.ld, a shuffle) waits like this: a lane that sees another role's abort while its neighbours see
// the phase complete must not leave them alone, and the fills and phases that a warp counts stay the same in all lanes.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err,
                                               uint64_t timeout_ns) {
    const uint32_t a = smem_u32(bar);
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(a, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(a, parity))) {
        const bool late = globaltimer_ns() - t0 > timeout_ns;
        if (__any_sync(0xFFFFFFFFu, late || *abort)) {
            if (late) {
                *abort = 1;
                atomicOr(err, kErrWaitTimeout);
            }
            __syncwarp();
            return false;
        }
    }
    return true;
}

// Lower bound of the deadline of a drain wait, independent of the (possibly very short) deadline of
// the ordinary waits: copies and MMAs in flight complete in microseconds, and a CTA must not exit
// (or free TMEM) before they have.
constexpr uint64_t kDrainFloorNs = 1000000000ull;

// Same, but ignores `abort` (used while draining in-flight copies and MMAs before exit). Waits at
// least kDrainFloorNs.
__device__ __forceinline__ bool mbar_wait_drain(uint64_t* bar, uint32_t parity, uint64_t timeout_ns) {
    const uint32_t a = smem_u32(bar);
    const uint64_t limit = timeout_ns > kDrainFloorNs ? timeout_ns : kDrainFloorNs;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(a, parity)) {
        if (globaltimer_ns() - t0 > limit) return false;
    }
    return true;
}

// Single-thread forms used on the drain path: one arrival that expects `bytes` more, and a
// completion of `bytes` without data (for copies that were never issued).
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// ---- shared / global vector access, tensor-map prefetch ---------------------------------------

__device__ __forceinline__ void st_shared_v4(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t saddr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr)
                 : "memory");
    return v;
}
// Streaming store (evict-first in L2): GEMM output is written once and not read back here, so it
// should not displace the operand tiles other CTAs are about to read from L2.
__device__ __forceinline__ void st_global_v4(void* p, const uint4& v) {
    asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void st_global_v8(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e,
                                             uint32_t f, uint32_t g, uint32_t h) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c),
                 "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---- tcgen05 ----------------------------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Waits for this thread's TMEM loads and ties the destination registers to the wait, so no use of
// them is scheduled above it.
template <int N>
__device__ __forceinline__ void reg_after_wait(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
template <int N>
__device__ __forceinline__ void tc_wait_ld_regs(uint32_t (&r)[N]) {
    tc_wait_ld();
    reg_after_wait(r);
}
template <int N>
__device__ __forceinline__ void tc_wait_ld_regs(uint32_t (&r0)[N], uint32_t (&r1)[N]) {
    tc_wait_ld();
    reg_after_wait(r0);
    reg_after_wait(r1);
}

// 32 lanes x 32 columns of 32-bit words: thread t of the warp gets lane (base_lane + t), columns
// [col, col + 32).
__device__ __forceinline__ void tc_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// 32 lanes x 16 columns of 32-bit words.
__device__ __forceinline__ void tc_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 32 lanes x 8 columns of 32-bit words.
__device__ __forceinline__ void tc_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// ---- CTA pairs (cluster of 2, cta_group::2) -----------------------------------------------------

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Shared::cluster address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t mapa_shared(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 32-bit load from a shared::cluster address (possibly in the peer CTA).
__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}
// Arrive on an mbarrier given by its shared::cluster address (possibly in the peer CTA), with the
// default CTA-scope release. The GEMM epilogue arrives this way to hand accumulator columns back to
// the MMA issuer; what must be ordered before the arrive are its TMEM loads, which tcgen05.wait::ld
// completes and tcgen05.fence::before_thread_sync orders. A cluster-scope release would also wait
// until the warp's earlier global stores of C are acknowledged, about 6k cycles per tile on the
// B200; the MMA issuer never reads C.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// ---- issue from a converged warp ------------------------------------------------------------------
// Every lane of the warp calls these together with the same arguments; elect.sync picks the one lane
// that executes the instruction. Keeping the issuing warp converged lets the operands live in
// uniform registers: issuing tcgen05 / TMA instructions from a single-lane branch instead was
// measured at 325 cycles per 128x256x32 MMA against 128 here (the MMA's own duration).

#define MX_ELECT_PRED "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t@e "

__device__ __forceinline__ void mbar_arrive_expect_tx_elect(uint64_t* bar, uint32_t bytes) {
    asm volatile(MX_ELECT_PRED "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d_elect(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t c0,
                                                  int32_t c1) {
    asm volatile(MX_ELECT_PRED
                 "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
                 "%4}], [%2];\n\t}" ::"r"(smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_load_elect(void* smem_dst, const void* gsrc, uint32_t bytes, uint64_t* bar) {
    asm volatile(MX_ELECT_PRED
                 "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(
                     smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair_elect(void* smem_dst, const CUtensorMap* map,
                                                       uint32_t bar_cluster_addr, int32_t c0, int32_t c1) {
    asm volatile(MX_ELECT_PRED
                 "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
                 "{%3, %4}], [%2];\n\t}" ::"r"(smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d_elect(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t c0,
                                                  int32_t c1, int32_t c2) {
    asm volatile(MX_ELECT_PRED
                 "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
                 "%4, %5}], [%2];\n\t}" ::"r"(smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair_elect(void* smem_dst, const CUtensorMap* map,
                                                       uint32_t bar_cluster_addr, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(MX_ELECT_PRED
                 "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
                 "{%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void tc_cp_elect(uint32_t taddr, uint64_t sdesc) {
    asm volatile(MX_ELECT_PRED "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc)
                 : "memory");
}
__device__ __forceinline__ void tc_cp_pair_elect(uint32_t taddr, uint64_t sdesc) {
    asm volatile(MX_ELECT_PRED "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc)
                 : "memory");
}
__device__ __forceinline__ void tc_mma_mxf8_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}
__device__ __forceinline__ void tc_mma_mxf8_pair_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                       uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}
// MXFP4: packed E2M1 operands, K = 64 per instruction, two E8M0 scales (blocks of 32) per row and instruction.
__device__ __forceinline__ void tc_mma_mxf4_pair_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                       uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}
// A whole MXFP4 stage (256 elements of K) under one election: per half of the stage the scale copies (A's and B's two
// row tiles' blocks; the second half's slot is 12 columns on) and two MMAs of 64 elements, then the commit on `bar` in
// both CTAs. Issued one by one, each with its own election, the issuing warp and not the tensor core set the pace:
// 5200 x 24576 x 4096 took 201 us (with a test before each MMA 230), like this, with the epilogue's direct stores, 190;
// all copies before all MMAs 192; the next stage's copies between this stage's MMAs 221.
// sda / sdb0 / sdb1: descriptors of the scale blocks of A and of B's row tiles in shared memory; the second block
// of each lies 512 bytes (32 descriptor units) behind the first.
__device__ __forceinline__ void tc_mxf4_stage_pair_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc0,
                                                         uint32_t idesc2, uint32_t sfa_t, uint64_t sda, uint64_t sdb0,
                                                         uint64_t sdb1, uint32_t accumulate, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 x, y;\n\t.reg .b32 b0, b1, a1, b2, b3, a0h, b0h, a1h, b2h;\n\t.reg .b16 m;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %9, 0;\n\tsetp.eq.b32 t, 0, 0;\n\tmov.b16 m, 3;\n\t"
        "add.u32 b0, %5, 4;\n\tadd.u32 b1, %5, 8;\n\tadd.u32 a1, %5, 12;\n\tadd.u32 b2, %5, 16;\n\tadd.u32 b3, %5, 20;\n\t"
        "or.b32 a0h, %5, 0x80000000;\n\tor.b32 b0h, b0, 0x80000000;\n\tor.b32 a1h, a1, 0x80000000;\n\tor.b32 b2h, b2, 0x80000000;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], %6;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [b0], %7;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [b1], %8;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [b0], p;\n\t"
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %4, [a0h], [b0h], t;\n\t"
        "add.s64 x, %6, 32;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [a1], x;\n\t"
        "add.s64 x, %7, 32;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [b2], x;\n\t"
        "add.s64 x, %8, 32;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [b3], x;\n\t"
        "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %3, [a1], [b2], t;\n\t"
        "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %4, [a1h], [b2h], t;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%10], m;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc0), "r"(idesc2), "r"(sfa_t), "l"(sda), "l"(sdb0), "l"(sdb1), "r"(accumulate),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tc_commit_elect(uint64_t* bar) {
    asm volatile(MX_ELECT_PRED "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                     smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_commit_pair_elect(uint64_t* bar, uint16_t cta_mask) {
    asm volatile(MX_ELECT_PRED
                 "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
                 "%1;\n\t}" ::"r"(smem_u32(bar)),
                 "h"(cta_mask)
                 : "memory");
}

// ---- UMMA descriptors --------------------------------------------------------------------------

// Shared-memory matrix descriptor, K-major operand tile written by TMA with the 128-byte swizzle:
// rows of 128 bytes, 8-row groups 1024 bytes apart (stride byte offset), descriptor version 1.
__device__ __forceinline__ uint64_t sdesc_kmajor_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1u) << 16;              // leading byte offset (unused for this layout)
    d |= static_cast<uint64_t>(1024u >> 4) << 32;      // stride byte offset: 8 rows x 128 B
    d |= static_cast<uint64_t>(1u) << 46;              // descriptor version (sm_100)
    d |= static_cast<uint64_t>(2u) << 61;              // 128-byte swizzle
    return d;
}

// Shared-memory descriptor for a 32-row x 16-byte scale block (no swizzle): rows 16 bytes apart,
// 8-row core matrices 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scale_block(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(128u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    return d;
}

// Instruction descriptor for kind::mxf8f6f4 with block scaling: E4M3 x E4M3, E8M0 scales, both
// operands K-major, M x N tile; sf_id picks the scale byte (the K-block of 32) inside each
// 32-bit TMEM scale word.
__host__ __device__ constexpr uint32_t idesc_mxf8_e4m3(uint32_t M, uint32_t N, uint32_t sf_id) {
    return (sf_id << 4)            // B scale-factor id
           | (0u << 7)             // A format: E4M3
           | (0u << 10)            // B format: E4M3
           | ((N >> 3) << 17)      // N / 8
           | (1u << 23)            // scale format: E8M0
           | ((M >> 4) << 24)      // M / 16
           | (sf_id << 29);        // A scale-factor id
}

// Instruction descriptor for kind::mxf4: E2M1 x E2M1 (format code 1), E8M0 scales, both operands K-major,
// K = 64; sf_id (0 or 2) picks the pair of scale bytes inside each 32-bit TMEM scale word. M is a multiple
// of 128.
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t M, uint32_t N, uint32_t sf_id) {
    return (sf_id << 4)            // B scale-factor id
           | (1u << 7)             // A format: E2M1
           | (1u << 10)            // B format: E2M1
           | ((N >> 3) << 17)      // N / 8
           | (1u << 23)            // scale format: E8M0
           | ((M >> 7) << 27)      // M / 128
           | (sf_id << 29);        // A scale-factor id
}

// ---- starting as the kernel in front ends -----------------------------------------------------------------
// A kernel launched with programmatic stream serialization may start as soon as the last blocks of the kernel in front
// of it have ended, before that one's writes are flushed and its end is seen by the host's queue (about 2 us between two
// eager launches). grid_wait() is its first statement, before any access to global memory and before TMEM is allocated:
// it waits until the kernel in front has ended and its writes are visible. So kernels do not overlap in what they read
// and write, and a chain of them stays ordered. Data that the kernel in front may have written is read with coherent
// loads only (no .nc: it asks for data that nothing writes during the kernel's life, which begins earlier here).
// No kernel lets the one behind start earlier than at its end (griddepcontrol.launch_dependents at its beginning): waiting
// blocks took places from working ones (router forward + backward, 5201 x 100: 17.9 us with it, 14.1 us without) and
// elsewhere it made no difference.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Coherent loads of data that is read once.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void ld_once_v8(const void* p, uint4& a, uint4& b) {
    asm volatile("ld.global.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}

}  // namespace mx
