// Tensor-core, tensor-memory and mbarrier helpers (inline PTX) of the kernels that multiply
// on the 5th-generation tensor cores: the sparse logits and the sparse attention.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "device.cuh"

namespace gkr {

namespace {

constexpr int kRowBytes = 128;           // one swizzle row: 64 bf16
constexpr int32_t kErrTimeout = 16;
constexpr uint64_t kWaitNs = 20000000;   // a wait gives up after 20 ms (a normal one takes us)

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// True once the phase with the given parity has completed.  A thread whose phase is not
// complete is suspended until it completes or kSuspendNs have passed: a waiting warp then
// takes no issue slots from the warps that work (spinning without the hint cost ~2 % of
// the sparse logits).  A build that defines GKR_WAIT_CLOCKS, for the tests of what happens then,
// has waits that run out: wait_quiet's limit is that many clocks, and a poll does not suspend.
#ifdef GKR_WAIT_CLOCKS
constexpr int64_t kWaitClocks = GKR_WAIT_CLOCKS;
constexpr uint32_t kSuspendNs = 0;
constexpr int kWaitPolls = 1;
#else
constexpr int64_t kWaitClocks = INT64_C(4000000000);   // 2 s at 2 GHz
constexpr uint32_t kSuspendNs = 20000;
constexpr int kWaitPolls = 64;
#endif
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return done != 0u;
}
__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Wait for the phase with the given parity to complete; false once kWaitNs have passed.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_ns() - t0 > kWaitNs) return false;
    return true;
}
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Make this thread's shared-memory stores visible to the tensor cores (async proxy).
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 inputs, fp32 accumulator; one thread.  A sits in
// tensor memory with row i in lane i and its K values two to a 32-bit column (the lower
// half holds the even k), so the K = 16 of one instruction span 8 columns.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the mbarrier once every tcgen05 operation this thread issued has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}
// 16 consecutive fp32 accumulator columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 consecutive 32-bit columns of this thread's lane (tcgen05.wait::st before handing
// them to the tensor cores).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint4 (&v)[4]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y),
        "r"(v[1].z), "r"(v[1].w), "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w),
        "r"(v[3].x), "r"(v[3].y), "r"(v[3].z), "r"(v[3].w)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor of a K-major operand with the 128-byte swizzle: start
// address >> 4 (bits 0-13), leading offset (unused by this layout; 1) at bits 16-29,
// stride between 8-row groups (1024 bytes) >> 4 at bits 32-45, descriptor version 1 at
// bits 46-47, swizzle mode 128B (2) at bits 61-63.  The operand's rows are 128 bytes (64
// bf16 of K); row r of an 8-row group sits at r * 128 in its 1024-byte group, and its
// 16-byte piece c at position c ^ r.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile(
        "{\n .reg .b64 state;\n mbarrier.arrive.shared::cta.b64 state, [%0];\n}\n" ::"r"(bar)
        : "memory");
}

// A wait that records a timeout instead of hanging: after the first failure the thread
// stops waiting (its results are discarded, see GKR_ERR_TIMEOUT).
__device__ __forceinline__ void wait_or_flag(uint32_t bar, uint32_t parity, bool& ok) {
    if (ok) ok = mbar_wait(bar, parity);
}

// The same for a whole warp: lane 0 waits, the warp follows it (__syncwarp orders the
// lanes' later accesses after lane 0's acquire); every lane gets the outcome.
__device__ __forceinline__ void warp_wait_or_flag(uint32_t bar, uint32_t parity, bool& ok,
                                                  int lane) {
    if (lane == 0) wait_or_flag(bar, parity, ok);
    ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
    __syncwarp();
}

// wait_or_flag for kernels whose warps run different code and wait at the same time: a poll is
// a few instructions, because the polls of waiting warps compete for issue slots and
// instruction fetches with the warps that work, and the limit is counted in SM clocks, which
// are read in a few cycles.  Who gave up (ok false) must neither arrive, issue, copy nor store
// on the strength of what it waited for: then nothing downstream completes either, and no result
// is written from data that did not come.
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, int64_t limit) {
    const int64_t t0 = clock64();
    do {
#pragma unroll 1
        for (int i = 0; i < kWaitPolls; ++i)
            if (mbar_try_wait(bar, parity)) return true;
    } while (clock64() - t0 <= limit);
    return false;
}
__device__ __forceinline__ void wait_quiet(uint32_t bar, uint32_t parity, bool& ok) {
    if (ok && !mbar_try_wait(bar, parity)) ok = mbar_wait_slow(bar, parity, kWaitClocks);
}
// The same for a converged warp, with one outcome: every lane waits, a vote decides.
__device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity) {
    const int64_t t0 = clock64();
    do {
#pragma unroll 1
        for (int i = 0; i < kWaitPolls; ++i)
            if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    } while (__all_sync(kFull, clock64() - t0 <= kWaitClocks));
    return false;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, bool& ok) {
    if (!__all_sync(kFull, mbar_try_wait(bar, parity))) ok = warp_wait_slow(bar, parity);
    return ok;
}
// The wait for copies and products that are under way when a CTA leaves: with the full limit in
// every build, and whatever gave up before.
__device__ __forceinline__ bool wait_landed(uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || mbar_wait_slow(bar, parity, INT64_C(4000000000));
}

// One arrival for a whole warp: every lane's earlier shared-memory writes (each lane has
// fenced them for the async proxy) are ordered before lane 0's arrive by __syncwarp.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link to the driver
// library); null when the driver does not provide it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// D[tmem] (+)= A[smem] * B[smem]^T of this CTA, bf16 inputs, fp32 accumulator; one thread.
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// ------------------------------------------------------------- CTA pairs (cta_group::2)
//
// Two CTAs of a cluster on neighbouring SMs multiply together: one thread of the leader (rank
// 0) issues tcgen05.mma for both, each CTA holding its rows of A and of D and half of B's
// columns, all at the same shared- and tensor-memory addresses in both.

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Address, in the cluster's shared window, of this CTA's `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// Arrive on an mbarrier anywhere in the cluster (a map_rank address).  What the arrivals of
// these kernels announce is read by the tensor cores of the arriving CTA's own SM, for which
// the writer has fenced it (fence_async_smem); no memory is handed from CTA to CTA, so the
// default release at CTA scope does.  (A release at cluster scope, and waits that acquire at it,
// cost a full memory barrier per arrival: the sparse attention's first form took 187 us so, 165
// us like this.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Have a tensor map (a kernel parameter) on hand before its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// TMA load of a 3-D box at (x, y, z) into this CTA's shared memory, counted on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
// One lane of a converged warp (warp-uniform code around it keeps addresses and descriptors in
// uniform registers, where tcgen05 wants them).
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}
// A descriptor with its lower half replaced.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t lo) {
    return (desc & 0xFFFFFFFF00000000u) | lo;
}
// D[tmem] (+)= A[smem] * B[smem]^T over the pair, bf16 inputs, fp32 accumulator; one thread.
__device__ __forceinline__ void mma_bf16_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// The same with A in tensor memory: K's values two to a column (the lower half the even k), 16
// of them in 8 columns, the CTA's 64 rows in lanes 0 .. 63 and again in lanes 64 .. 127.
__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// Arrive on the mbarrier at this offset in both CTAs once every tcgen05 operation the elected
// lane issued has completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar, uint32_t elected) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;\n}" ::"r"(bar),
        "h"(static_cast<uint16_t>(3)), "r"(elected)
        : "memory");
}
// 32 consecutive 32-bit columns of this thread's lane; tcgen05.wait::ld before their use.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];\n tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]),
        "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]),
        "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]),
        "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
// Descriptor of an operand whose reduction runs over its 128-byte rows (MN-major, 128-byte
// swizzle): 64 elements of M or N to a row, 8 rows (of K) to a 1024-byte group.  `block`:
// bytes between blocks of 64 elements of M or N (bits 16-29); the groups of K follow each
// other at 1024 bytes (bits 32-45).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t block) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
           (static_cast<uint64_t>(block >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

}  // namespace
}  // namespace gkr
