// Sparse decode attention over MXFP4 records (272 B), softmax and value product included.
//
// Operation (FlashMLA overview page, DSA section: a decode query attends to the entries its
// index row lists, -1 marking an invalid one; the 512-dim latent row is key and value of every
// head): for query i and head h, with K[k] the bf16 row kv_gather returns for indices[i, k],
//   s[k] = sm_scale * q[i, h] . K[k],  m = max s,  l = sum exp(s - m) over the valid entries,
//   out[i, h] = sum exp(s[k] - m) K[k] / l,   lse[i, h] = m + log l;
// a query without a valid entry gets zeros and -inf.  With weights,
//   weights[i, k] += sum over h of exp(s[k] - lse[i, h])
// for the valid entries, the attention that record received.
//
// One pass over the records with a running maximum and sum, the tensor cores of two SMs on one
// query.  Per record and 128 heads both products are 2 x 128 x 512 multiply-adds, 16 cycles of
// two SMs' tensor cores, against 272 bytes of memory: with many heads the products bound
// the kernel, so everything else is arranged to stay below those 16 cycles.
//   * The accumulator of a query, 128 heads x 512 dims fp32, is all of an SM's tensor memory.  A
//     pair of CTAs (cta_group::2, M = 128) splits it: each holds its 64 heads' rows, 256 columns
//     on 128 lanes, and has room for the logits.
//   * Records are dequantised once to bf16 in shared memory and are there both operands: rows
//     of 128 bytes (64 dims) in 8-row swizzle groups read K-major for q . K (reduction over
//     dims) and MN-major for p . K (reduction over records).  A product of the pair takes half
//     of its columns from each CTA, so for q . K a CTA needs 32 of a chunk's 64 records in
//     full (32 KB), for p . K all 64 in its half of the dims (32 KB), a quarter in common.  The
//     operand's address has to be the same in both CTAs, so a stage of 32 KB is filled twice:
//     first with the CTA's 32 records; once q . K has read them, the half of the dims that
//     the other CTA multiplies is replaced by the other 32 records' dims of its own half.  While
//     that happens the softmax of the chunk runs.
//   * Work: the chunks of all queries in a row, cut evenly over the pairs.  A query that lies
//     inside one pair's run is finished there; the pieces of a cut one go to the workspace
//     (fp32 rows and their log-sum-exp) and a second kernel joins them.
#include <cmath>
#include <mutex>
#include <vector>

#include "decode.cuh"
#include "device.cuh"
#include "launch.h"
#include "tensor.cuh"

namespace gkr {

namespace {

constexpr int32_t kErrIndex = 4;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

constexpr int kPairHeads = 64;           // heads (rows) of each CTA of the pair
constexpr int kChunkKeys = 64;           // records per chunk
constexpr int kOwnKeys = 32;             // of which a CTA dequantises this many in full
constexpr int kStages = 4;               // chunks in flight
constexpr int kSoftmaxWarps = 4;         // warps 0..3: warp w owns tensor-memory lanes 32w ..
constexpr int kProducerWarps = 8;        // warps 4..11: gather and dequantise
constexpr int kMmaWarp = kSoftmaxWarps + kProducerWarps;    // warp 12: products (rank 0)
constexpr int kLoadWarp = kMmaWarp + 1;                     // warp 13: query tiles
constexpr int kAttendThreads = (kLoadWarp + 1) * 32;
constexpr uint32_t kBlockBytes = kOwnKeys * kRowBytes;      // 64 dims of the stage's 32 rows
constexpr uint32_t kHalfBytes = 4 * kBlockBytes;            // 256 dims
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kQBlockBytes = kPairHeads * kRowBytes;   // 64 dims of the query tile
constexpr uint32_t kQBytes = 8 * kQBlockBytes;
constexpr uint32_t kPBytes = kPairHeads * kRowBytes;        // probabilities of a chunk, bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;          // logits: two buffers of 32 columns; output at 0
// A new maximum replaces the running one only when it is this much larger (in powers of two):
// probabilities then stay below 2^8, and the accumulator is rarely rescaled.
constexpr float kLag = 8.0f;
// Probabilities are taken as exp2(s - m + kLift): bf16 ends at 2^-133, and without the lift terms
// that the output still shows (it ends there too) would be rounded away before they are
// multiplied by a record's values and summed.  At most 2^24 with kLag, far from overflow.
constexpr float kLift = 16.0f;

// kind::f16 over the pair, M = 128, fp32 accumulator, bf16 A and B (fields as in logits.cu):
// logits N = 64, both K-major; output N = 256, B MN-major (bit 16).
constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
constexpr uint32_t kIdescS = idesc(kChunkKeys, false);
constexpr uint32_t kIdescO = idesc(256, true);

// The cut of a call's chunks over the pairs: pair g takes chunks [total * g / pairs,
// total * (g + 1) / pairs) of the queries' chunks taken one query after another.
struct Cut {
    int64_t per_query;   // chunks of a query, >= 1
    int64_t total;
    int32_t pairs;
    __host__ __device__ int64_t begin(int64_t g) const { return total * g / pairs; }
    __host__ __device__ int64_t owner(int64_t chunk) const { return ((chunk + 1) * pairs - 1) / total; }
};

// Shared memory of a CTA, from a 1024-byte boundary.
constexpr uint32_t kOffStages = kQBytes;
constexpr uint32_t kOffP = kOffStages + kStages * kStageBytes;
constexpr uint32_t kOffMax = kOffP + 2 * kPBytes;           // [2][128] row maxima
constexpr uint32_t kOffSum = kOffMax + 2 * 128 * 4;         // [128] row sums
constexpr uint32_t kOffBars = kOffSum + 128 * 4;

struct alignas(8) PairBarriers {
    // in the leader: arrivals of both CTAs
    uint64_t full_k[kStages];    // producers: the chunk's records are in place for q . K
    uint64_t full_v[kStages];    // producers: ... and for p . K
    uint64_t p_full[2];          // softmax: the logits are read, the probabilities written
    uint64_t q_full;             // the query tiles have arrived
    // in each CTA
    uint64_t s_full[2];          // products: the logits of a chunk are complete
    uint64_t stage_empty[kStages];   // products: p . K has read the stage
    uint64_t o_done[2];          // products: p . K of a chunk is complete
    uint64_t q_free;             // products: q . K of a query's last chunk is complete
    uint64_t q_tma;              // this CTA's query tile has arrived
    uint32_t tmem_base;
    int32_t timed_out;
};
constexpr size_t kAttendSmem = 1024 + kOffBars + sizeof(PairBarriers);
static_assert(kAttendSmem <= 227 * 1024, "a CTA's shared memory");

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One lane's part of a record: 32 dims, their scale byte.
struct Unit {
    uint4 codes;
    uint32_t scale;
};

// Unit u of the record in slot idx; zeros (the value 0) for an entry that is none.
__device__ __forceinline__ Unit load_unit(const AttentionParams& p, const uint8_t* base,
                                          int32_t row, int u) {
    Unit r;
    r.codes = make_uint4(0u, 0u, 0u, 0u);
    r.scale = 0u;
    if (base != nullptr) {
        r.codes = ldg_na16(base + row * 256 + u * 16);
        r.scale = ldg_u8(base + static_cast<int64_t>(p.block_size) * 256 + row * 16 + u);
    }
    return r;
}
// The page (null: no entry) and row of slot idx.
__device__ __forceinline__ const uint8_t* record_page(const AttentionParams& p, int32_t idx,
                                                      int32_t& row) {
    row = 0;
    if (idx < 0 || idx >= p.num_slots) return nullptr;
    uint32_t page, r;
    page_row(static_cast<uint32_t>(idx), static_cast<uint32_t>(p.block_size), page, r);
    row = static_cast<int32_t>(r);
    return p.cache + static_cast<int64_t>(page) * p.page_stride;
}
// The unit's 32 bf16 values into row r of a block of 64 dims: 16-byte pieces c0 .. c0 + 3.
__device__ __forceinline__ void store_unit(uint8_t* block, int r, int c0, const Unit& t) {
    uint8_t* const row = block + (r >> 3) * 1024 + (r & 7) * kRowBytes;
    const uint32_t w[4] = {t.codes.x, t.codes.y, t.codes.z, t.codes.w};
    if (__builtin_expect(t.scale <= kE2m1OneStepByte, 1)) {
        const uint32_t f = e2m1_factor(t.scale);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st16(row + (((c0 + j) ^ (r & 7)) << 4), dequant8_e2m1_scaled(w[j], f));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st16(row + (((c0 + j) ^ (r & 7)) << 4), dequant8_e2m1(w[j], t.scale));
    }
}

// Eight fp32 values, scaled, as bf16.
__device__ __forceinline__ uint4 pack8(const float* v, float f) {
    return make_uint4(pack_bf16x2_rn(__fmul_rn(v[0], f), __fmul_rn(v[1], f)),
                      pack_bf16x2_rn(__fmul_rn(v[2], f), __fmul_rn(v[3], f)),
                      pack_bf16x2_rn(__fmul_rn(v[4], f), __fmul_rn(v[5], f)),
                      pack_bf16x2_rn(__fmul_rn(v[6], f), __fmul_rn(v[7], f)));
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const AttentionParams p, const Cut cut, const __grid_constant__ CUtensorMap q_map) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    PairBarriers* const bars = reinterpret_cast<PairBarriers*>(smem + kOffBars);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t pair = blockIdx.x >> 1;
    const int64_t c0 = cut.begin(pair);
    const int n = static_cast<int>(cut.begin(pair + 1) - c0);   // chunks of this pair, >= 1

    if (warp == kMmaWarp) {
        tmem_alloc_pair(smem_addr(&bars->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&bars->full_k[s]), 2 * kProducerWarps);
            mbar_init(smem_addr(&bars->full_v[s]), 2 * kProducerWarps);
            mbar_init(smem_addr(&bars->stage_empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&bars->p_full[b]), 2 * kSoftmaxWarps);
            mbar_init(smem_addr(&bars->s_full[b]), 1);
            mbar_init(smem_addr(&bars->o_done[b]), 1);
        }
        mbar_init(smem_addr(&bars->q_full), 2);
        mbar_init(smem_addr(&bars->q_free), 1);
        mbar_init(smem_addr(&bars->q_tma), 1);
        bars->timed_out = 0;
        mbar_init_fence();
    }
    pdl_wait_previous();
    pdl_release_next();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();   // the other CTA's barriers exist
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    bool ok = true;

    // chunk j of this pair: query and chunk within it, counted
    int64_t qi = c0 / cut.per_query;
    int64_t ci = c0 - qi * cut.per_query;

    if (warp >= kSoftmaxWarps && warp < kMmaWarp) {
        // ------------------------------------------------------------- producers
        // A lane handles one of the CTA's 32 records (row r) and one of the other CTA's (row r
        // too): two units of the first, one of the second.  Eight lanes of a store have eight
        // rows of one swizzle group, so their pieces fall into different banks; the four
        // lanes of a record read 64 contiguous bytes.
        const int pw = warp - kSoftmaxWarps;
        const int r = (pw & 3) * 8 + (lane & 7);
        const int u_own = (pw >> 2) * 8 + (lane >> 3);                      // and + 4
        const int u_oth = static_cast<int>(rank) * 8 + (pw >> 2) * 4 + (lane >> 3);
        const int k_own = static_cast<int>(rank) * kOwnKeys + r;
        const int k_oth = (1 - static_cast<int>(rank)) * kOwnKeys + r;
        // blocks of 64 dims hold two units
        const uint32_t own_a = (u_own >> 1) * kBlockBytes, own_b = own_a + 2 * kBlockBytes;
        const int c_own = (u_own & 1) * 4, c_oth = (u_oth & 1) * 4;
        // the half of the stage whose dims the other CTA multiplies
        const uint32_t oth = (rank == 0 ? kHalfBytes : 0u) +
                             ((u_oth - static_cast<int>(rank) * 8) >> 1) * kBlockBytes;
        const uint32_t full_k = map_rank(smem_addr(&bars->full_k[0]), 0);
        const uint32_t full_v = map_rank(smem_addr(&bars->full_v[0]), 0);

        // indices of chunk j, the records of chunks j - 1 and j - 2 on their way
        int32_t i_own = -1, i_oth = -1, i_oth2 = -1;
        int j_idx = 0;
        auto next_indices = [&]() {
            i_oth2 = i_oth;
            i_own = i_oth = -1;
            if (j_idx < n) {
                const int32_t* const row = p.indices + qi * p.index_stride;
                const int64_t k = ci * kChunkKeys;
                if (k + k_own < p.topk) i_own = __ldg(row + k + k_own);
                if (k + k_oth < p.topk) i_oth = __ldg(row + k + k_oth);
                if (++ci == cut.per_query) {
                    ci = 0;
                    ++qi;
                }
            }
            ++j_idx;
        };
        Unit a, b, o;         // being stored: chunk j + 1's own units, chunk j's other
        Unit na, nb, no;      // on their way: one chunk later
        auto load_own = [&](int32_t idx) {
            int32_t row;
            const uint8_t* const base = record_page(p, idx, row);
            na = load_unit(p, base, row, u_own);
            nb = load_unit(p, base, row, u_own + 4);
        };
        auto load_oth = [&](int32_t idx) {
            int32_t row;
            const uint8_t* const base = record_page(p, idx, row);
            no = load_unit(p, base, row, u_oth);
        };
        next_indices();       // chunk 0
        load_own(i_own);
        a = na;
        b = nb;
        next_indices();       // chunk 1
        o = Unit{};
#pragma unroll 1
        for (int j = -1; j < n; ++j) {
            load_own(i_own);                       // chunk j + 2
            load_oth(i_oth2);                      // chunk j + 1
            next_indices();                        // chunk j + 3
            if (j + 1 < n) {
                const int s = (j + 1) & (kStages - 1);
                if (j + 1 >= kStages)
                    warp_wait_or_flag(smem_addr(&bars->stage_empty[s]),
                                      (((j + 1) / kStages) - 1) & 1, ok, lane);
                uint8_t* const st = smem + kOffStages + s * kStageBytes;
                store_unit(st + own_a, r, c_own, a);
                store_unit(st + own_b, r, c_own, b);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(full_k + 8 * s);
            }
            if (j >= 0) {
                const int s = j & (kStages - 1);
                warp_wait_or_flag(smem_addr(&bars->s_full[j & 1]), (j >> 1) & 1, ok, lane);
                store_unit(smem + kOffStages + s * kStageBytes + oth, r, c_oth, o);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(full_v + 8 * s);
            }
            a = na;
            b = nb;
            o = no;
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------- query tiles
        if (lane == 0) {
            uint32_t loads = 0;
            for (int j = 0; j < n; ++j) {
                if (j == 0 || ci == 0) {
                    // the tile may go once the last chunk of the query before is multiplied
                    if (j > 0) wait_or_flag(smem_addr(&bars->q_free), (loads - 1) & 1, ok);
                    const uint32_t bar = smem_addr(&bars->q_tma);
                    if (ok) {
                        mbar_expect_tx(bar, kQBytes);
                        for (int kb = 0; kb < 8; ++kb)
                            tma_load_3d(smem_addr(smem) + kb * kQBlockBytes, &q_map, bar, 64 * kb,
                                        static_cast<int32_t>(rank) * kPairHeads,
                                        static_cast<int32_t>(qi));
                        wait_or_flag(bar, loads & 1, ok);
                    }
                    ++loads;
                    mbar_arrive_cluster(map_rank(smem_addr(&bars->q_full), 0));
                }
                if (++ci == cut.per_query) {
                    ci = 0;
                    ++qi;
                }
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------- products
        if (lane == 0 && rank == 0) {
            const uint64_t q_desc = sw128_desc(smem_addr(smem));
            uint32_t loads = 0;
            bool first = true;    // chunk j - 1 opens its query in this pair
            auto output = [&](int j, bool fresh) {
                const int s = j & (kStages - 1);
                wait_or_flag_cluster(smem_addr(&bars->full_v[s]), (j / kStages) & 1, ok);
                wait_or_flag_cluster(smem_addr(&bars->p_full[j & 1]), (j >> 1) & 1, ok);
                tc_fence_after_sync();
                const uint64_t a = sw128_desc(smem_addr(smem + kOffP + (j & 1) * kPBytes));
                const uint64_t b = sw128_mn_desc(smem_addr(smem + kOffStages + s * kStageBytes),
                                                 kBlockBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k) {        // 16 records
#pragma unroll
                    for (int d = 0; d < 2; ++d) {    // 128 of each CTA's 256 dims
                        const uint32_t off = (k >> 1) * kHalfBytes + (k & 1) * 2048 + d * 2 * kBlockBytes;
                        mma_bf16_ss_pair(tmem + 128 * d, a + 2 * k, b + (off >> 4), kIdescO,
                                         (fresh && k == 0) ? 0u : 1u);
                    }
                }
                mma_commit_pair(smem_addr(&bars->stage_empty[s]));
                mma_commit_pair(smem_addr(&bars->o_done[j & 1]));
            };
            for (int j = 0; j < n; ++j) {
                const bool opens = j == 0 || ci == 0;
                if (opens) {   // finish the query before, then wait for the new one's tile
                    if (j > 0) output(j - 1, first);
                    wait_or_flag_cluster(smem_addr(&bars->q_full), loads & 1, ok);
                    ++loads;
                }
                const int s = j & (kStages - 1);
                wait_or_flag_cluster(smem_addr(&bars->full_k[s]), (j / kStages) & 1, ok);
                tc_fence_after_sync();
                const uint64_t b = sw128_desc(smem_addr(smem + kOffStages + s * kStageBytes));
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    mma_bf16_ss_pair(tmem + kSCol + 32 * (j & 1),
                                     q_desc + (((k >> 2) * kQBlockBytes + (k & 3) * 32) >> 4),
                                     b + (((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4), kIdescS,
                                     k != 0 ? 1u : 0u);
                mma_commit_pair(smem_addr(&bars->s_full[j & 1]));
                if (++ci == cut.per_query) {
                    ci = 0;
                    if (j + 1 < n) mma_commit_pair(smem_addr(&bars->q_free));
                }
                if (!opens) output(j - 1, first);
                first = opens;
            }
            output(n - 1, first);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------- softmax, epilogue
        // Lane L of the 128: head L % 64 of this CTA; of a chunk the records of CTA L / 64; of
        // the output the dims 256 (L / 64) ...  The two lanes of a head exchange their maxima.
        const int row = (warp & 1) * 32 + lane;
        const int half = warp >> 1;
        const int head = static_cast<int>(rank) * kPairHeads + row;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        float* const maxima = reinterpret_cast<float*>(smem + kOffMax);
        float* const sums = reinterpret_cast<float*>(smem + kOffSum);
        const int self = half * 64 + row, peer = self ^ 64;
        const uint32_t p_full = map_rank(smem_addr(&bars->p_full[0]), 0);
        const float scale = __fmul_rn(p.sm_scale, kLog2e);   // logits in powers of two
        auto pair_sync = [&]() {   // the two warps that share their heads
            asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory");
        };
        auto index_of = [&](int64_t q, int64_t c) -> int32_t {
            const int64_t k = c * kChunkKeys + half * kOwnKeys + lane;
            return k < p.topk ? __ldg(p.indices + q * p.index_stride + k) : -1;
        };
        bool bad = false;
        float m = -INFINITY, l = 0.0f;
        bool fresh = true;         // no chunk of this query is in the accumulator
        int64_t seg = ci;          // the segment's first chunk
        int32_t idx = index_of(qi, ci);
        for (int j = 0; j < n; ++j) {
            const bool is = idx >= 0 && idx < p.num_slots;
            bad |= !is && idx != -1;
            const uint32_t live = __ballot_sync(kFull, is);
            const bool last = j + 1 == n || ci + 1 == cut.per_query;   // of this segment
            if (j + 1 < n) idx = ci + 1 == cut.per_query ? index_of(qi + 1, 0) : index_of(qi, ci + 1);
            warp_wait_or_flag(smem_addr(&bars->s_full[j & 1]), (j >> 1) & 1, ok, lane);
            tc_fence_after_sync();
            float v[32];
            tmem_ld32(tmem + lanes + kSCol + 32 * (j & 1), v);
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                v[i] = (live >> i) & 1u ? __fmul_rn(v[i], scale) : -INFINITY;
                top = fmaxf(top, v[i]);
            }
            maxima[(j & 1) * 128 + self] = top;
            pair_sync();
            top = fmaxf(top, maxima[(j & 1) * 128 + peer]);
            const bool rise = top > m + kLag || (m == -INFINITY && top > m);
            if (__any_sync(kFull, rise)) {
                const float fix = rise ? exp2_approx(__fsub_rn(m, top)) : 1.0f;
                if (rise) m = top;
                l = __fmul_rn(l, fix);
                if (!fresh) {
                    // the products of the chunk before are in the accumulator
                    warp_wait_or_flag(smem_addr(&bars->o_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, ok,
                                      lane);
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        float t[32];
                        tmem_ld32(tmem + lanes + c, t);
#pragma unroll
                        for (int i = 0; i < 32; ++i) t[i] = __fmul_rn(t[i], fix);
                        tmem_st32(tmem + lanes + c, t);
                    }
                    tmem_st_wait();
                }
            }
            const float ref = m == -INFINITY ? 0.0f : __fsub_rn(m, kLift);
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                v[i] = exp2_approx(__fsub_rn(v[i], ref));
                sum[i & 3] = __fadd_rn(sum[i & 3], v[i]);
            }
            l = __fadd_rn(l, __fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3])));
            // the buffer's last reader, the value product of chunk j - 2
            if (j >= 2)
                warp_wait_or_flag(smem_addr(&bars->o_done[j & 1]), ((j >> 1) - 1) & 1, ok, lane);
            uint8_t* const prow = smem + kOffP + (j & 1) * kPBytes + (row >> 3) * 1024 +
                                  (row & 7) * kRowBytes;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                st16(prow + (((half * 4 + c) ^ (row & 7)) << 4), pack8(v + 8 * c, 1.0f));
            fence_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(p_full + 8 * (j & 1));
            fresh = false;
            if (last) {
                sums[self] = l;
                pair_sync();
                const float total = __fadd_rn(half == 0 ? l : sums[peer], half == 0 ? sums[peer] : l);
                pair_sync();   // read before the next segment's sums
                warp_wait_or_flag(smem_addr(&bars->o_done[j & 1]), (j >> 1) & 1, ok, lane);
                tc_fence_after_sync();
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                const bool whole = seg == 0 && ci + 1 == cut.per_query;
                const float lse2 = total == 0.0f ? -INFINITY : __fadd_rn(__fsub_rn(m, kLift), log2f(total));
                const bool mine = head < p.num_heads && ok;
                if (whole) {
                    uint8_t* const out = static_cast<uint8_t*>(p.out) +
                                         (qi * p.num_heads + head) * 1024 + half * 512;
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        float t[32];
                        tmem_ld32(tmem + lanes + c, t);
                        if (mine) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                st16(out + 2 * c + 16 * i,
                                     total == 0.0f ? make_uint4(0u, 0u, 0u, 0u) : pack8(t + 8 * i, inv));
                        }
                    }
                    if (mine && half == 0)
                        p.lse[qi * p.num_heads + head] = __fmul_rn(lse2, kLn2);
                } else {
                    // a piece that does not begin its query is its pair's first: slot 0
                    const int64_t slot = 2 * pair + (seg == 0 ? 1 : 0);
                    float* const rows = static_cast<float*>(p.workspace);
                    float* const dst = rows + (slot * p.num_heads + head) * 512 + half * 256;
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        float t[32];
                        tmem_ld32(tmem + lanes + c, t);
                        if (mine) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<float4*>(dst + c + i) =
                                    total == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                                  : make_float4(__fmul_rn(t[i], inv), __fmul_rn(t[i + 1], inv),
                                                                __fmul_rn(t[i + 2], inv), __fmul_rn(t[i + 3], inv));
                        }
                    }
                    if (mine && half == 0)
                        rows[2 * static_cast<int64_t>(cut.pairs) * p.num_heads * 512 +
                             slot * p.num_heads + head] = lse2;
                }
                tc_fence_before_sync();
                m = -INFINITY;
                l = 0.0f;
                fresh = true;
                seg = 0;
            }
            if (++ci == cut.per_query) {
                ci = 0;
                ++qi;
            }
        }
        if (rank == 0 && (warp == 0 || warp == 2) && __any_sync(kFull, bad) && lane == 0)
            report(p.err, kErrIndex);
    }
    if (!ok) atomicOr(&bars->timed_out, 1);
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && bars->timed_out != 0) report(p.err, kErrTimeout);
    cluster_sync();   // no CTA leaves while the other's products or arrivals reach it
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// Joins the pieces of each cut query: out = sum_i exp2(lse_i - lse) rows_i.  A block of 128
// threads takes one head, four dims a thread, of the query that pair g's run begins inside of,
// if g is the second pair on it.
__global__ void __launch_bounds__(128) join_kernel(const AttentionParams p, const Cut cut) {
    const int64_t g = 1 + blockIdx.x / p.num_heads;
    const int head = static_cast<int>(blockIdx.x % p.num_heads);
    pdl_wait_previous();
    pdl_release_next();
    const int64_t qi = cut.begin(g) / cut.per_query;
    const int64_t g0 = cut.owner(qi * cut.per_query);
    if (g != g0 + 1) return;
    const int64_t g1 = cut.owner((qi + 1) * cut.per_query - 1);
    if (g1 == g0) return;   // finished by its pair
    const float* const rows = static_cast<const float*>(p.workspace);
    const float* const lses = rows + 2 * static_cast<int64_t>(cut.pairs) * p.num_heads * 512 + head;
    // the first piece ends its pair's run (slot 1), the others begin theirs (slot 0)
    auto slot = [&](int64_t i) -> int64_t { return 2 * i + (i == g0 ? 1 : 0); };
    float m = -INFINITY;
    for (int64_t i = g0; i <= g1; ++i) m = fmaxf(m, lses[slot(i) * p.num_heads]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
#pragma unroll 4
    for (int64_t i = g0; i <= g1; ++i) {
        const float w = exp2_approx(__fsub_rn(lses[slot(i) * p.num_heads], ref));
        const float4 t = *reinterpret_cast<const float4*>(
            rows + (slot(i) * p.num_heads + head) * 512 + 4 * threadIdx.x);
        sum = __fadd_rn(sum, w);
        acc.x = __fmaf_rn(w, t.x, acc.x);
        acc.y = __fmaf_rn(w, t.y, acc.y);
        acc.z = __fmaf_rn(w, t.z, acc.z);
        acc.w = __fmaf_rn(w, t.w, acc.w);
    }
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    const uint2 v = make_uint2(pack_bf16x2_rn(__fmul_rn(acc.x, inv), __fmul_rn(acc.y, inv)),
                               pack_bf16x2_rn(__fmul_rn(acc.z, inv), __fmul_rn(acc.w, inv)));
    const int64_t at = qi * p.num_heads + head;
    st8(static_cast<uint8_t*>(p.out) + at * 1024 + 8 * threadIdx.x, v);
    if (threadIdx.x == 0)
        p.lse[at] = sum == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, log2f(sum)), kLn2);
}

constexpr int kHeadsPerBlock = 8;
constexpr int kTile = 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, d));
    return v;
}
// Records k0 .. k0 + 31 of query qi as bf16 rows of 1024 bytes in `rows` (zeros for an entry
// that is none); returns the bits of the valid ones.  Every thread of the block calls it.
__device__ __forceinline__ uint32_t load_tile(const AttentionParams& p, int64_t qi, int64_t k0,
                                              uint8_t* rows, uint32_t* valid, int warp, int lane) {
    __syncthreads();   // the previous tile has been read
    if (threadIdx.x == 0) *valid = 0;
    __syncthreads();
    for (int r = warp; r < kTile; r += kHeadsPerBlock) {
        const int64_t k = k0 + r;
        const int32_t idx = k < p.topk ? __ldg(p.indices + qi * p.index_stride + k) : -1;
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (idx >= 0 && idx < p.num_slots) {
            uint32_t page, row;
            page_row(static_cast<uint32_t>(idx), static_cast<uint32_t>(p.block_size), page, row);
            const uint8_t* const base = p.cache + static_cast<int64_t>(page) * p.page_stride;
            const uint32_t* const data =
                reinterpret_cast<const uint32_t*>(base + static_cast<int64_t>(row) * 256);
            const uint8_t* const sc = base + static_cast<int64_t>(p.block_size) * 256 + row * 16;
            a = dequant8_e2m1(__ldg(data + lane), __ldg(sc + (lane >> 2)));
            b = dequant8_e2m1(__ldg(data + 32 + lane), __ldg(sc + 8 + (lane >> 2)));
            if (lane == 0) atomicOr(valid, 1u << r);
        } else if (idx != -1 && lane == 0) {
            report(p.err, kErrIndex);
        }
        st16(rows + r * 1024 + 16 * lane, a);
        st16(rows + r * 1024 + 512 + 16 * lane, b);
    }
    __syncthreads();
    return *valid;
}

// This lane's 16 dims of a row's dot product with x, summed over the warp.
__device__ __forceinline__ float dot(const float (&x)[16], const uint8_t* row, int lane) {
    float v[16];
    unpack_bf16x8(lds16(row + 16 * lane), v);
    unpack_bf16x8(lds16(row + 512 + 16 * lane), v + 8);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s = __fmaf_rn(x[i], v[i], s);
    return warp_sum(s);
}

__device__ __forceinline__ void load_head(const AttentionParams& p, int64_t qi, int h, int lane,
                                          float (&x)[16]) {
    const uint8_t* const row = static_cast<const uint8_t*>(p.q) + (qi * p.num_heads + h) * 1024;
    unpack_bf16x8(*reinterpret_cast<const uint4*>(row + 16 * lane), x);
    unpack_bf16x8(*reinterpret_cast<const uint4*>(row + 512 + 16 * lane), x + 8);
}

// weights[qi, k] += sum over the heads of exp(s - lse): the logits once more, now that each
// head's lse is known; a block takes 32 entries of a query, a warp every eighth head.
__global__ void __launch_bounds__(kHeadsPerBlock * 32) weight_kernel(const AttentionParams p,
                                                                     const int64_t tiles) {
    __shared__ __align__(16) uint8_t rows[kTile * 1024];
    __shared__ uint32_t valid;
    __shared__ float part[kHeadsPerBlock][32];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t qi = blockIdx.x / tiles;
    const int64_t k0 = (blockIdx.x - qi * tiles) * kTile;
    pdl_wait_previous();
    pdl_release_next();
    const uint32_t live = load_tile(p, qi, k0, rows, &valid, warp, lane);
    const float scale = __fmul_rn(p.sm_scale, kLog2e);
    float sum = 0.0f;
    for (int h = warp; h < p.num_heads; h += kHeadsPerBlock) {
        float x[16];
        load_head(p, qi, h, lane, x);
        const float lse = __fmul_rn(p.lse[qi * p.num_heads + h], kLog2e);
        float s = -INFINITY;
        for (int k = 0; k < kTile; ++k) {
            const float d = dot(x, rows + k * 1024, lane);
            if (lane == k && ((live >> k) & 1u) != 0u) s = __fmul_rn(d, scale);
        }
        if (((live >> lane) & 1u) != 0u) sum = __fadd_rn(sum, exp2_approx(__fsub_rn(s, lse)));
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && ((live >> lane) & 1u) != 0u) {
        float t = part[0][lane];
        for (int w = 1; w < kHeadsPerBlock; ++w) t = __fadd_rn(t, part[w][lane]);
        float* const dst = p.weights + qi * p.weight_stride + k0 + lane;
        *dst = __fadd_rn(*dst, t);
    }
}

// The pairs of CTAs that the current device holds at once (cached per device).
struct PairCount {
    int device;
    int32_t pairs;
};
std::mutex g_pairs_mutex;
std::vector<PairCount> g_pairs;

cudaError_t resident_pairs(int32_t* pairs) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_pairs_mutex);
    for (const PairCount& c : g_pairs) {
        if (c.device == dev) {
            *pairs = c.pairs;
            return cudaSuccess;
        }
    }
    e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kAttendSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = kAttendSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, attend_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    g_pairs.push_back({dev, n});
    *pairs = n;
    return cudaSuccess;
}

cudaError_t make_cut(int64_t num_queries, int64_t topk, Cut* cut) {
    int32_t pairs = 0;
    const cudaError_t e = resident_pairs(&pairs);
    if (e != cudaSuccess) return e;
    cut->per_query = topk == 0 ? 1 : (topk + kChunkKeys - 1) / kChunkKeys;
    cut->total = num_queries * cut->per_query;
    cut->pairs = static_cast<int32_t>(cut->total < pairs ? cut->total : pairs);
    return cudaSuccess;
}

// Whether some query is cut, so that there are pieces to join.
bool has_pieces(const Cut& cut) {
    for (int32_t g = 1; g < cut.pairs; ++g)
        if (cut.begin(g) % cut.per_query != 0) return true;
    return false;
}

// The queries [num_queries, num_heads, 512] as a 3-D tensor map with boxes of 64 dims x 64
// heads and the 128-byte swizzle; heads past num_heads read as zeros.
cudaError_t q_tensor_map(const AttentionParams& p, CUtensorMap* map) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {512, static_cast<cuuint64_t>(p.num_heads),
                                static_cast<cuuint64_t>(p.num_queries)};
    const cuuint64_t strides[2] = {1024, static_cast<cuuint64_t>(1024) * p.num_heads};
    const cuuint32_t box[3] = {64, kPairHeads, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r =
        encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box,
               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t attention_workspace(int32_t num_heads, int64_t num_queries, int64_t topk,
                                int64_t* bytes) {
    Cut cut;
    const cudaError_t e = make_cut(num_queries, topk, &cut);
    if (e != cudaSuccess) return e;
    // two pieces a pair: a row and a log-sum-exp for each head
    *bytes = has_pieces(cut) ? 2 * static_cast<int64_t>(cut.pairs) * num_heads * (512 + 1) * 4 : 0;
    return cudaSuccess;
}

cudaError_t launch_sparse_attention(const AttentionParams& p, cudaStream_t stream) {
    Cut cut;
    cudaError_t e = make_cut(p.num_queries, p.topk, &cut);
    if (e != cudaSuccess) return e;
    CUtensorMap map;
    e = q_tensor_map(p, &map);
    if (e != cudaSuccess) return e;
    e = launch_kernel(attend_kernel, 2 * static_cast<int64_t>(cut.pairs), kAttendThreads, kAttendSmem,
                      stream, p.pdl, p, cut, map);
    if (e != cudaSuccess) return e;
    if (has_pieces(cut)) {
        e = launch_kernel(join_kernel, static_cast<int64_t>(cut.pairs - 1) * p.num_heads, 128, 0,
                          stream, p.pdl, p, cut);
        if (e != cudaSuccess) return e;
    }
    if (p.weights == nullptr || p.topk == 0) return e;
    const int64_t tiles = (p.topk + kTile - 1) / kTile;
    return launch_kernel(weight_kernel, p.num_queries * tiles, kHeadsPerBlock * 32, 0, stream,
                         p.pdl, p, tiles);
}

}  // namespace gkr
