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
// two SMs' tensor cores, against 272 bytes of memory: with many heads the products are the
// floor, so everything else is arranged to run beside them.
//   * The accumulator of a query, 128 heads x 512 dims fp32, is all of an SM's tensor memory.  A
//     pair of CTAs (cta_group::2, M = 128) splits it: each holds its 64 heads' rows, 256 columns
//     on 128 lanes, and has room for two chunks' logits and for three quarters of the query,
//     which so need not be read from shared memory by every product.
//   * Records come by 16-byte asynchronous copies of three warps, their slots six chunks ahead: a
//     chunk takes about 2000 cycles, a load from memory up to 4000.  (By the copy engine's
//     four-row gathers, 90 cycles each, they came too slowly: 79 us where this took 75.5.)
//   * They are dequantised once to bf16 in shared memory and are there both operands: rows
//     of 128 bytes (64 dims) in 8-row swizzle groups read K-major for q . K (reduction over
//     dims) and MN-major for p . K (reduction over records).  A product of the pair takes half
//     of its columns from each CTA, so for q . K a CTA needs 32 of a chunk's 64 records in
//     full (32 KB), for p . K all 64 in its half of the dims (32 KB), a quarter in common.  The
//     operand's address has to be the same in both CTAs, so a stage of 32 KB is filled twice:
//     first with the CTA's 32 records; once q . K has read them, the half of the dims that
//     the other CTA multiplies is replaced by the other 32 records' dims of its own half.  While
//     that happens the softmax of the chunk runs.
//   * Work: the chunks of all queries in a row, cut evenly over the pairs, or whole queries
//     where that costs no more (make_cut).  A query that lies inside one pair's run is
//     finished there; the pieces of a cut one go to the workspace (fp32 rows and their
//     log-sum-exp) and a second kernel joins them.  Where a run of one query were too long for one
//     accumulator, the cut is over more pairs than the device holds at once (kRunChunks).
// Measured: 128 queries x 128 heads x 2048 entries 76.8 us, 895 TFLOP/s, 46 % of the measured
// matrix rate.  A chunk of 64 records takes 2000 cycles, its products alone 1165 (64 columns a
// product run at 63 % of the rate of 256).  What is left is shared out: issue slots are 70 %
// taken, the warp that issues the products, the warps that dequantise and those that gather each
// spend nearly all of a chunk's time on it, and speeding up one of them alone moves little.
// Tried: a warp for each product (slower by itself, 72 registers; as fast with two gathering
// warps); eight warps that replace (82 us); the dequantisation's warps on alternate chunks
// (78.5), with a fourth stage in the place of the next query's blocks 73, but 4 to 7 % slower for
// short lists; 32 rows of each CTA for up to 64 heads, every second softmax warp idle: as fast.
#include <cmath>

#include "attend.cuh"
#include "device.cuh"
#include "launch.h"
#include "tensor.cuh"

namespace gkr {

namespace {

constexpr int kPairHeads = 64;           // heads (rows) of each CTA of the pair
constexpr int kChunkKeys = 64;           // records per chunk
constexpr int kOwnKeys = 32;             // of which a CTA dequantises this many in full
constexpr int kStages = 3;               // chunks of dequantised records in flight
constexpr int kRawStages = 3;            // chunks of raw records in flight
constexpr int kSoftmaxWarps = 8;         // warps 0..7: warp w has tensor-memory lanes 32 (w % 4) ..
                                         // and half w / 4 of their columns
constexpr int kOwnWarps = 8;             // dequantise the CTA's own records for q . K
constexpr int kRefillWarps = 4;          // dequantise the other CTA's records for p . K
constexpr int kFirstOwn = kSoftmaxWarps;
constexpr int kFirstRefill = kFirstOwn + kOwnWarps;
constexpr int kMmaWarp = kFirstRefill + kRefillWarps;       // products (rank 0)
constexpr int kGatherWarps = 3;          // raw records: own in two halves, the others' half
constexpr int kFirstGather = kMmaWarp + 1;
constexpr int kIndexRing = 8;            // chunks of indices (kept as many) a gather warp holds,
constexpr int kIndexAhead = 6;           // and has on their way
constexpr int kAttendThreads = (kFirstGather + kGatherWarps) * 32;   // 24 warps: up to 80 registers (16 bytes spilled)
constexpr uint32_t kBlockBytes = kOwnKeys * kRowBytes;      // 64 dims of the stage's 32 rows
constexpr uint32_t kHalfBytes = 4 * kBlockBytes;            // 256 dims
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kQBlockBytes = kPairHeads * kRowBytes;   // 64 dims of the query tile
constexpr int kQTmemBlocks = 6;          // blocks of 64 dims of the query in tensor memory
constexpr uint32_t kQBytes = (8 - kQTmemBlocks) * kQBlockBytes;   // and in shared memory
constexpr uint32_t kPBytes = kPairHeads * kRowBytes;        // probabilities of a chunk, bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;          // logits: two buffers of 32 columns; output at 0
constexpr uint32_t kQCol = 320;          // the query's first 384 dims, two to a column
static_assert(kQCol + kQTmemBlocks * 32 <= kTmemCols, "tensor memory");
// kind::f16 over the pair, M = 128, fp32 accumulator, bf16 A and B (fields as in logits.cu):
// logits N = 64, both K-major; output N = 256, B MN-major (bit 16).
constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
constexpr uint32_t kIdescS = idesc(kChunkKeys, false);
constexpr uint32_t kIdescO = idesc(256, true);

// The cut of a call's chunks over the pairs: pair g takes chunks [total * g / pairs,
// total * (g + 1) / pairs) of the queries' chunks taken one query after another, or, with
// `each` > 0, `each` whole queries.
struct Cut {
    int64_t per_query;   // chunks of a query, >= 1
    int64_t total;
    int64_t each;
    int32_t pairs;
    __host__ __device__ int64_t begin(int64_t g) const {
        const int64_t b = each > 0 ? each * per_query * g : total * g / pairs;
        return b < total ? b : total;
    }
    // The pair that takes a chunk, where the cut is even: the last g with total * g / pairs < chunk + 1.
    __device__ int64_t pair_of(int64_t chunk) const { return ((chunk + 1) * pairs - 1) / total; }
};
// Chunks of a query that one accumulator sums, at most.  The tensor cores cut off what a sum of theirs cannot hold, all in
// one direction, on average half of its last bit for every 16 records: over a million records results came out
// 0.4 % too small, over 131072 it is 0.08 %.  Longer queries are cut over more pairs than the device holds at once.
constexpr int64_t kRunChunks = 2048;

// Shared memory of a CTA, from a 1024-byte boundary.
constexpr uint32_t kOffNext = kQBytes;                      // the next query's first blocks
constexpr uint32_t kOffStages = kOffNext + kQTmemBlocks * kQBlockBytes;
constexpr uint32_t kOffP = kOffStages + kStages * kStageBytes;
constexpr uint32_t kOffRaw = kOffP + 2 * kPBytes;
// raw stage: the codes of the 32 own records in two blocks of 32 rows of 128 bytes (one for each
// half of the dims), those of the other CTA's 32 records in this CTA's half in a third, all with
// the 128-byte swizzle (eight rows' pieces lie in different banks); then the scale rows
constexpr uint32_t kRawBlock = kOwnKeys * 128;
constexpr uint32_t kRawOth = 2 * kRawBlock;
constexpr uint32_t kRawOwnScales = kRawOth + kRawBlock;
constexpr uint32_t kRawOthScales = kRawOwnScales + kOwnKeys * 16;
constexpr uint32_t kRawBytes = kRawOthScales + kOwnKeys * 16;
constexpr uint32_t kOffMax = kOffRaw + kRawStages * kRawBytes;   // [4][64] maxima of a head
constexpr uint32_t kOffSum = kOffMax + 256 * 4;             // [4][64] sums of a head
constexpr uint32_t kOffIndex = kOffSum + 256 * 4;           // [gather warp][kIndexRing][32]
constexpr uint32_t kOffLive = kOffIndex + kGatherWarps * kIndexRing * 128;   // [kIndexRing][CTA] masks
constexpr uint32_t kOffBars = kOffLive + kIndexRing * 2 * 4;
static_assert(kRawStages + kStages + 1 < kIndexRing && kIndexAhead < kIndexRing,
              "the softmax reads a chunk's masks before they are replaced");

struct alignas(8) PairBarriers {
    // in the leader: arrivals of both CTAs
    uint64_t full_k[kStages];    // own warps: the chunk's records are in place for q . K
    uint64_t p_full[2];          // refill warps: ... and for p . K; softmax: the logits are read,
                                 // the probabilities written
    uint64_t q_full;             // softmax: a query is in place for q . K
    // in each CTA
    uint64_t q_next;             // the next query's first blocks are in shared memory
    uint64_t q_live;             // this query's last blocks are
    uint64_t raw_own[kRawStages], raw_own_empty[kRawStages];   // raw records: landed, read
    uint64_t raw_oth[kRawStages], raw_oth_empty[kRawStages];
    uint64_t s_full[2];          // products: the logits of a chunk are complete
    uint64_t stage_empty[kStages];   // products: p . K of a chunk is complete, its stage read
    uint64_t live[kIndexRing];   // gather warps: both masks of a chunk's entries are written
    uint64_t drained;            // products: every one that was issued is complete
    uint32_t next_loads, live_loads;   // of the query, issued so far (q_next, q_live)
    uint32_t tmem_base;
    volatile int32_t timed_out;  // a wait of this CTA gave up
};
constexpr size_t kAttendSmem = 1024 + kOffBars + sizeof(PairBarriers);
static_assert(kAttendSmem <= 227 * 1024, "a CTA's shared memory");

// A unit's 32 dims (16 bytes of codes, a scale byte) as bf16 into four 16-byte pieces of a
// swizzled row: piece j of the unit lies at the first one's address with j in bits 4 and 5
// flipped.
__device__ __forceinline__ void store_unit(uint32_t codes, uint32_t scale, uint32_t out) {
    const uint4 c = lds16_at(codes);
    uint32_t s;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s) : "r"(scale) : "memory");
    const uint32_t f = e2m1_factor(s);
    sts16(out, dequant8_e2m1(c.x, f));
    sts16(out ^ 16u, dequant8_e2m1(c.y, f));
    sts16(out ^ 32u, dequant8_e2m1(c.z, f));
    sts16(out ^ 48u, dequant8_e2m1(c.w, f));
}

// Named barriers of the warps of one role: one or two threads wait on the mbarriers, the others here,
// where a waiting warp takes no issue slots.  Instruction supply bounds a kernel of so many roles
// before anything else does: with every warp polling for itself and each role's loop unrolled
// in full, the warps ran 11200 instructions a chunk and missed the instruction cache on 17 % of
// its requests.  So the waits are few, the loops short, and roles that do the same share
// their code.  The waiting threads sit in warps on other schedulers than the one that
// issues the products.
constexpr int kPollThread = 32;   // of the softmax warps
constexpr int kOwnBar = 1, kRefillBar = 2, kSoftmaxBar = 3, kHeadsBar = 4;   // and 5
// The wait of a thread that polls for a group of dequantising warps.  Should it give up, it keeps the
// group at its named barrier until the warp that issues the products has left (`drained`; it
// misses the group's arrivals and gives up in turn): only then may stages be overwritten and
// barriers be arrived at out of turn.  (To tell the group, so that it does neither, took 3 % more
// time for every call, by a flag or by the barrier.)
__device__ __noinline__ bool wait_slow_or_hold(uint32_t bar, uint32_t parity, uint32_t drained) {
    if (mbar_wait_slow(bar, parity, kWaitClocks)) return true;
    for (int i = 0; i < 3; ++i)   // its wait may have begun later, and then it drains
        if (wait_landed(drained, 0)) break;
    return false;
}
__device__ __forceinline__ void wait_or_hold(uint32_t bar, uint32_t parity, uint32_t drained, bool& ok) {
    if (ok && !mbar_try_wait(bar, parity)) ok = wait_slow_or_hold(bar, parity, drained);
}

// Row `row` of a query tile (blocks of 64 rows of 64 dims, 128-byte swizzle) into this thread's
// lane of tensor memory at `dst`.  A is read by the tensor cores from both halves of the lanes,
// each of which produces half of the columns, so both hold every row.
// This call moves blocks `first` .. `first` + 2.
__device__ __forceinline__ void query_to_tmem(uint32_t tile, int row, int first, uint32_t dst) {
    const uint32_t src = tile + row * kRowBytes + ((row & 7) << 4);
#pragma unroll 1
    for (int b = first; b < first + kQTmemBlocks / 2; ++b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // 32 dims
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lds16_at((src ^ ((4 * h + i) << 4)) + b * kQBlockBytes);
            tmem_st16(dst + 32 * b + 16 * h, v);
        }
    }
    tmem_st_wait();
}

// kParted: part of a prefix attention, with a prefix in front of the lists or fp32 rows as results, divided by
// the sum of the probabilities as rounded, as the tiles' are (a form of its own, as the tests for them
// cost the plain one 1 to 3 %, and its results stay what they were).
template <bool kParted>
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
            mbar_init(smem_addr(&bars->full_k[s]), 2 * kOwnWarps);
            mbar_init(smem_addr(&bars->stage_empty[s]), 1);
        }
        for (int s = 0; s < kRawStages; ++s) {
            mbar_init(smem_addr(&bars->raw_own[s]), 2 * 32);   // lanes of two warps
            mbar_init(smem_addr(&bars->raw_oth[s]), 32);
            mbar_init(smem_addr(&bars->raw_own_empty[s]), kOwnWarps);
            mbar_init(smem_addr(&bars->raw_oth_empty[s]), kRefillWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&bars->p_full[b]), 2 * (kSoftmaxWarps + kRefillWarps));
            mbar_init(smem_addr(&bars->s_full[b]), 1);
        }
        for (int i = 0; i < kIndexRing; ++i) mbar_init(smem_addr(&bars->live[i]), 2);
        mbar_init(smem_addr(&bars->q_full), 2 * kSoftmaxWarps);
        mbar_init(smem_addr(&bars->q_next), 1);
        mbar_init(smem_addr(&bars->q_live), 1);
        mbar_init(smem_addr(&bars->drained), 1);
        bars->next_loads = 0;
        bars->live_loads = 0;
        bars->timed_out = 0;
        mbar_init_fence();
    }
    if (threadIdx.x == kPollThread) prefetch_map(&q_map);
    pdl_wait_previous();
    pdl_release_next();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();   // the other CTA's barriers exist
    tc_fence_after_sync();
    // All 512 columns are this CTA's, so they begin at address 0: a constant, which keeps the
    // products' addresses in uniform registers.
    constexpr uint32_t tmem = 0;
    bool ok = bars->tmem_base == 0;

    // chunk j of this pair: query and chunk within it, counted
    int64_t qi = c0 / cut.per_query;
    int64_t ci = c0 - qi * cut.per_query;

    if (warp >= kFirstOwn && warp < kMmaWarp) {
        // ------------------------------------------------------------- dequantisation
        // Eight warps put the CTA's own records, in full, into a stage for q . K; four replace
        // the half of it whose dims the other CTA multiplies by the other records' half.  Both
        // run the same instructions (see kOwnBar).  A lane takes two units of 32 dims of record
        // r.  Eight lanes have eight rows of one swizzle group, so what they load and what
        // they store lies in different banks.
        const bool own = warp < kFirstRefill;
        const int w = own ? warp - kFirstOwn : warp - kFirstRefill;
        const int r = (w & 3) * 8 + (lane & 7);
        const int u = (w >> 2) * 8 + (lane >> 3);           // and + 4: two blocks of 64 dims on
        const uint32_t src = (own ? (w >> 2) * kRawBlock : kRawOth) + r * 128 +
                             (((lane >> 3) ^ (r & 7)) << 4);
        const uint32_t src_s = (own ? kRawOwnScales : kRawOthScales + rank * 8) + r * 16 + u;
        const uint32_t dst = kOffStages + (own || rank != 0 ? 0u : kHalfBytes) +
                             (u >> 1) * kBlockBytes + r * kRowBytes + (((u & 1) * 4 ^ (r & 7)) << 4);
        const uint32_t full = map_rank(smem_addr(own ? &bars->full_k[0] : &bars->p_full[0]), 0);
        const uint32_t raw_full = smem_addr(own ? &bars->raw_own[0] : &bars->raw_oth[0]);
        const uint32_t raw_empty = smem_addr(own ? &bars->raw_own_empty[0] : &bars->raw_oth_empty[0]);
        const uint32_t raw0 = smem_addr(smem + kOffRaw);
        const uint32_t out0 = smem_addr(smem) + dst;
        const int bar = own ? kOwnBar : kRefillBar, threads = own ? kOwnWarps * 32 : kRefillWarps * 32;
        Ring<kStages> st;
        Ring<kRawStages> rw;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            // two threads wait, each for one thing: one after the other takes 200 cycles more
            if (w == 2 && lane == 0) {
                wait_or_hold(raw_full + 8 * rw.s, rw.parity, smem_addr(&bars->drained), ok);
            } else if (w == 3 && lane == 0 && (!own || j >= kStages)) {
                // the stage is free; q . K has read what is replaced
                wait_or_hold(own ? smem_addr(&bars->stage_empty[st.s]) : smem_addr(&bars->s_full[j & 1]),
                             own ? st.parity ^ 1u : (j >> 1) & 1, smem_addr(&bars->drained), ok);
            }
            group_sync(bar, threads);
            const uint32_t raw = raw0 + rw.s * kRawBytes, out = out0 + st.s * kStageBytes;
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
                store_unit(raw + (src ^ (h << 6)), raw + src_s + 4 * h, out + h * 2 * kBlockBytes);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(raw_empty + 8 * rw.s);
                mbar_arrive_cluster(full + 8 * (own ? st.s : j & 1));
            }
            st.next();
            rw.next();
        }
    } else if (warp >= kFirstGather) {
        // ------------------------------------------------------------- raw records
        // Three warps run this: one for each half of the own records' dims, one for this CTA's
        // half of the others'.  The indices come into a ring in shared memory six chunks ahead
        // (a global load takes more than a chunk's time), lane i decodes record i of the
        // chunk's 32, eight lanes copy a half-row of 128 bytes, and every lane its record's 16
        // scale bytes; zeros for an entry that is none.  (The copy engine's four-row gathers take
        // 90 cycles each, 24 of them a chunk: at 2150 cycles they set the pace.)
        const int g = warp - kFirstGather;
        const bool own = g < 2;
        const uint32_t cta = own ? rank : 1u - rank;        // whose records
        const int key = static_cast<int>(cta) * kOwnKeys + lane;
        const uint32_t full = smem_addr(own ? &bars->raw_own[0] : &bars->raw_oth[0]);
        const uint32_t empty = smem_addr(own ? &bars->raw_own_empty[0] : &bars->raw_oth_empty[0]);
        const uint32_t raw0 = smem_addr(smem + kOffRaw);
        const int sub = lane >> 3, piece = lane & 7;        // row 4 i + sub, 16 bytes of it
        const uint8_t* const src = p.cache + (own ? g : rank) * 128 + 16 * piece;
        // rows 4 i + sub and 8 bytes of a swizzle group: i flips bit 2 of the row
        const uint32_t dst = g * kRawBlock + sub * 128 + ((piece ^ sub) << 4);
        const uint32_t scale_dst = (own ? kRawOwnScales : kRawOthScales) + 16 * lane;
        const uint32_t ring = smem_addr(smem + kOffIndex) + g * kIndexRing * 128 + 4 * lane;
        int ahead = 0;                                      // the next chunk to fetch indices of
        auto fetch = [&]() {
            if (ahead < n) {
                const uint32_t to = ring + (ahead & (kIndexRing - 1)) * 128;
                const int64_t k = ci * kChunkKeys + key;
                if (k < p.topk)
                    cp_async4(to, !kParted              ? p.indices + qi * p.index_stride + k
                                  : k < p.prefix_length ? p.prefix + k
                                                        : p.indices + qi * p.index_stride + (k - p.prefix_length));
                else asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(-1) : "memory");
                if (++ci == cut.per_query) {
                    ci = 0;
                    ++qi;
                }
                ++ahead;
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kIndexAhead; ++i) fetch();
        bool bad = false;
        Ring<kRawStages> rw;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            cp_async_wait<kIndexAhead - 1>();               // chunk j's indices are here
            int32_t idx;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(idx) : "r"(ring + (j & (kIndexRing - 1)) * 128) : "memory");
            const bool is = idx >= 0 && idx < p.num_slots;
            bad |= !is && idx != -1;
            const uint32_t live = __ballot_sync(kFull, is);
            uint32_t page, r;
            page_row(is ? static_cast<uint32_t>(idx) : 0u, static_cast<uint32_t>(p.block_size), page, r);
            const int64_t at = static_cast<int64_t>(page) * p.page_stride;
            const int32_t row = is ? static_cast<int32_t>(at >> 8) + static_cast<int32_t>(r) : -1;   // of 256 bytes
            if (j >= kRawStages && !warp_wait(empty + 8 * rw.s, rw.parity ^ 1u, ok)) break;
            const uint32_t raw = raw0 + rw.s * kRawBytes, bar = full + 8 * rw.s;
            if (g != 1) {
                if (lane == 0) {
                    reinterpret_cast<uint32_t*>(smem + kOffLive)[(j & (kIndexRing - 1)) * 2 + cta] = live;
                    mbar_arrive(smem_addr(&bars->live[j & (kIndexRing - 1)]));
                }
                cp_async16_or_zeros(raw + scale_dst,
                                    p.cache + at + static_cast<int64_t>(p.block_size) * 256 + r * 16u, is);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int32_t from = __shfl_sync(kFull, row, 4 * i + sub);
                cp_async16_or_zeros(raw + (dst ^ ((i & 1) << 6)) + i * 512,
                                    src + static_cast<int64_t>(from < 0 ? 0 : from) * 256, from >= 0);
            }
            cp_async_arrive(bar);
            fetch();
            rw.next();
        }
        if (g != 1 && rank == 0 && __any_sync(kFull, bad) && lane == 0) report(p.err, kErrIndex);
        cp_async_wait<0>();   // the copies in flight land before the CTA leaves
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------- products
        // The whole warp runs this, one lane issues (elect_lane).
        if (rank == 0) {
            const uint32_t elected = elect_lane();
            const uint64_t q_desc = sw128_desc(smem_addr(smem));
            const uint64_t k_desc0 = sw128_desc(smem_addr(smem + kOffStages));
            const uint64_t v_desc0 = sw128_mn_desc(smem_addr(smem + kOffStages), kBlockBytes);
            const uint64_t p_desc0 = sw128_desc(smem_addr(smem + kOffP));
            const uint32_t q_lo = static_cast<uint32_t>(q_desc), k_lo = static_cast<uint32_t>(k_desc0);
            const uint32_t v_lo = static_cast<uint32_t>(v_desc0), p_lo = static_cast<uint32_t>(p_desc0);
            uint32_t loads = 0;
            Ring<kStages> sk, sv;
            // q . K runs one chunk ahead of p . K within a query; jq, jo: their next chunks,
            // ci and co: those within the query
            int64_t co = ci;
            bool fresh = true;    // chunk jo opens its query in this pair
            int jq = 0, jo = 0;
#pragma unroll 1
            while (jo < n) {
                const bool opens = jq == 0 || ci == 0;
                if (jq < n && jq - jo < 2 && !(opens && jo < jq)) {
                    if (opens) {
                        if (!warp_wait(smem_addr(&bars->q_full), loads & 1, ok)) break;
                        ++loads;
                    }
                    if (!warp_wait(smem_addr(&bars->full_k[sk.s]), sk.parity, ok)) break;
                    tc_fence_after_sync();
                    const uint32_t d = tmem + kSCol + 32 * (jq & 1);
                    // one addition a product: the lower half of the descriptor (start addresses
                    // stay below 2^14 sixteen-byte units, so nothing carries), the rest constant
                    const uint32_t b = k_lo + sk.s * (kStageBytes >> 4);
                    if (elected) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {       // 16 dims
                            const uint64_t bk = desc_at(k_desc0, b + (((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4));
                            if (k < 4 * kQTmemBlocks)
                                mma_bf16_ts_pair(d, tmem + kQCol + 8 * k, bk, kIdescS, k != 0);
                            else
                                mma_bf16_ss_pair(d, desc_at(q_desc, q_lo + ((((k >> 2) - kQTmemBlocks) * kQBlockBytes + (k & 3) * 32) >> 4)),
                                                 bk, kIdescS, true);
                        }
                    }
                    __syncwarp();
                    mma_commit_pair(smem_addr(&bars->s_full[jq & 1]), elected);
                    if (++ci == cut.per_query) ci = 0;
                    sk.next();
                    ++jq;
                } else {
                    if (!warp_wait(smem_addr(&bars->p_full[jo & 1]), (jo >> 1) & 1, ok)) break;
                    tc_fence_after_sync();
                    const uint32_t a = p_lo + (jo & 1) * (kPBytes >> 4);
                    const uint32_t b = v_lo + sv.s * (kStageBytes >> 4);
                    if (elected) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {            // 16 records; k / 2: of which CTA
#pragma unroll
                            for (int h = 0; h < 2; ++h)          // 128 of each CTA's 256 dims
                                mma_bf16_ss_pair(tmem + 128 * h, desc_at(p_desc0, a + 2 * k),
                                                 desc_at(v_desc0, b + (((k >> 1) * kHalfBytes + (k & 1) * 2048 +
                                                                        h * 2 * kBlockBytes) >> 4)),
                                                 kIdescO, k != 0 || !fresh);
                        }
                    }
                    __syncwarp();
                    mma_commit_pair(smem_addr(&bars->stage_empty[sv.s]), elected);
                    sv.next();
                    ++jo;
                    fresh = false;
                    if (++co == cut.per_query) {
                        co = 0;
                        fresh = true;
                    }
                }
            }
            // whatever ended the loop, no product is under way when the pair leaves
            mma_commit_pair(smem_addr(&bars->drained), elected);
            if (!wait_landed(smem_addr(&bars->drained), 0)) ok = false;
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------- softmax, epilogue
        // Tensor-memory lane L: head L % 64 of this CTA; of a chunk the records of CTA L / 64; of
        // the output the dims 256 (L / 64) ...  Two warps share a lane, one for each half of its
        // columns (records, dims), so four threads have a head; they exchange maxima and sums.
        const int quarter = warp & 3, part = warp >> 2;
        const int row = (warp & 1) * 32 + lane;
        const int half = quarter >> 1;
        const int head = static_cast<int>(rank) * kPairHeads + row;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        float* const maxima = reinterpret_cast<float*>(smem + kOffMax) + row;
        float* const sums = reinterpret_cast<float*>(smem + kOffSum) + row;
        const int self = (part * 2 + half) * 64;
        const uint32_t p_full = map_rank(smem_addr(&bars->p_full[0]), 0);
        const float scale = __fmul_rn(p.sm_scale, kLog2e);   // logits in powers of two
        // the warps of a head; whether any of their threads says so
        auto head_sync = [&]() { group_sync(kHeadsBar + (warp & 1), 128); };
        auto head_any = [&](bool mine) -> bool { return group_any(kHeadsBar + (warp & 1), 128, mine); };
        const uint32_t q_full = map_rank(smem_addr(&bars->q_full), 0);
        // A query's first 384 dims wait in shared memory since the query before was moved, and go
        // to tensor memory; the last 128 come straight to where q . K reads them.
        const int64_t q_last = (c0 + n - 1) / cut.per_query;
        uint32_t q_parity = 0;
        auto fetch_next = [&](int64_t q) {   // one thread
            ++bars->next_loads;
            mbar_expect_tx(smem_addr(&bars->q_next), kQTmemBlocks * kQBlockBytes);
#pragma unroll 1
            for (int b = 0; b < kQTmemBlocks; ++b)
                tma_load_3d(smem_addr(smem) + kOffNext + b * kQBlockBytes, &q_map,
                            smem_addr(&bars->q_next), 64 * b, static_cast<int32_t>(rank) * kPairHeads,
                            static_cast<int32_t>(q));
        };
        auto query = [&](int64_t q) {
            if (threadIdx.x == kPollThread && ok) {
                ++bars->live_loads;
                mbar_expect_tx(smem_addr(&bars->q_live), kQBytes);
#pragma unroll 1
                for (int b = kQTmemBlocks; b < 8; ++b)
                    tma_load_3d(smem_addr(smem) + (b - kQTmemBlocks) * kQBlockBytes, &q_map,
                                smem_addr(&bars->q_live), 64 * b, static_cast<int32_t>(rank) * kPairHeads,
                                static_cast<int32_t>(q));
                wait_quiet(smem_addr(&bars->q_next), q_parity, ok);
            }
            group_sync(kSoftmaxBar, kSoftmaxWarps * 32);
            query_to_tmem(smem_addr(smem) + kOffNext, row, part * kQTmemBlocks / 2, tmem + lanes + kQCol);
            fence_async_smem();   // what was read is read, before the copy engine writes there
            tc_fence_before_sync();
            group_sync(kSoftmaxBar, kSoftmaxWarps * 32);
            if (threadIdx.x == kPollThread && ok) {
                if (q < q_last) fetch_next(q + 1);
                wait_quiet(smem_addr(&bars->q_live), q_parity, ok);
            }
            ok = __all_sync(kFull, ok) != 0;   // one outcome a warp, the polling thread's with it
            if (lane == 0 && ok) mbar_arrive_cluster(q_full);
            q_parity ^= 1u;
        };
        if (threadIdx.x == kPollThread && ok) fetch_next(qi);
        query(qi);
        float m = -INFINITY, l = 0.0f, rounded = 0.0f;   // rounded: see the tiles' softmax (kParted)
        bool fresh = true;         // no chunk of this query is in the accumulator
        int64_t seg = ci;          // the segment's first chunk
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const bool last = j + 1 == n || ci + 1 == cut.per_query;   // of this segment
            // the other CTA's records are not part of what q . K waits for, so their mask has a
            // barrier of its own (the ring's next round comes after this chunk's probabilities)
            if (ok) warp_wait(smem_addr(&bars->live[j & (kIndexRing - 1)]), (j / kIndexRing) & 1, ok);
            const uint32_t live =
                (reinterpret_cast<const uint32_t*>(smem + kOffLive)[(j & (kIndexRing - 1)) * 2 + half] >>
                 (16 * part)) & 0xFFFFu;
            // q . K of this chunk is complete, and with it, issued before, p . K of chunk j - 2:
            // the probabilities' buffer is free
            if (ok) warp_wait(smem_addr(&bars->s_full[j & 1]), (j >> 1) & 1, ok);
            tc_fence_after_sync();
            float v[16];
            tmem_ld16(tmem + lanes + kSCol + 32 * (j & 1) + 16 * part, v);
            const uint64_t scale2 = f32x2(scale, scale);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                f32x2_split(mul_f32x2(f32x2(v[i], v[i + 1]), scale2), v[i], v[i + 1]);
            if (live != 0xFFFFu) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (((live >> i) & 1u) == 0u) v[i] = -INFINITY;
            }
            float top = fmaxf(v[0], v[1]);
#pragma unroll
            for (int i = 2; i < 16; i += 2) top = fmaxf(top, fmaxf(v[i], v[i + 1]));
            // Rarely a logit is far above its head's reference; the head's four threads learn of
            // it by the barrier alone, and only then exchange their maxima.
            if (head_any(top > m + kLag || (m == -INFINITY && top > m))) {
                maxima[self] = top;
                head_sync();
                top = fmaxf(fmaxf(maxima[0], maxima[64]), fmaxf(maxima[128], maxima[192]));
                head_sync();   // read before they are written again
                const bool rise = top > m + kLag || (m == -INFINITY && top > m);
                const float root = rise ? exp2_approx(__fmul_rn(__fsub_rn(m, top), 0.5f)) : 1.0f;
                if (rise) m = top;
                l = __fmul_rn(l, __fmul_rn(root, root));
                if constexpr (kParted) rounded = __fmul_rn(rounded, __fmul_rn(root, root));
                if (!fresh) {
                    // the products of the chunk before are in the accumulator
                    if (ok) warp_wait(smem_addr(&bars->stage_empty[(j - 1) % kStages]), ((j - 1) / kStages) & 1, ok);
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int i = 0; i < 256; i += 32) {   // the columns twice, a factor each time
                        const int c = 128 * part + (i & 127);
                        float t[32];
                        tmem_ld32(tmem + lanes + c, t);
#pragma unroll
                        for (int k = 0; k < 32; ++k) t[k] = __fmul_rn(t[k], root);
                        tmem_st32(tmem + lanes + c, t);
                        tmem_st_wait();
                    }
                }
            }
            const float ref = m == -INFINITY ? 0.0f : __fsub_rn(m, kLift);
            const uint64_t ref2 = f32x2(-ref, -ref);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                f32x2_split(add_f32x2(f32x2(v[i], v[i + 1]), ref2), v[i], v[i + 1]);
                v[i] = exp2_flush(v[i]);
                v[i + 1] = exp2_flush(v[i + 1]);
            }
            uint64_t sum2 = add_f32x2(f32x2(v[0], v[1]), f32x2(v[2], v[3]));
#pragma unroll
            for (int i = 4; i < 16; i += 4)
                sum2 = add_f32x2(sum2, add_f32x2(f32x2(v[i], v[i + 1]), f32x2(v[i + 2], v[i + 3])));
            float sum_a, sum_b;
            f32x2_split(sum2, sum_a, sum_b);
            l = __fadd_rn(l, __fadd_rn(sum_a, sum_b));
            const uint32_t prow = smem_addr(smem + kOffP) + (j & 1) * kPBytes + row * kRowBytes +
                                  ((half * 4 + part * 2 ^ (row & 7)) << 4);
            const uint4 w0 = pack8(v), w1 = pack8(v + 8);
            sts16(prow, w0);
            sts16(prow ^ 16u, w1);
            fence_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive_cluster(p_full + 8 * (j & 1));
            if constexpr (kParted) {
                f32x2_split(add_f32x2(sum_rounded(w0), sum_rounded(w1)), sum_a, sum_b);
                rounded = __fadd_rn(rounded, __fadd_rn(sum_a, sum_b));
            }
            fresh = false;
            if (last) {
                // q . K of this query is complete: the next one may take its place, and is
                // multiplied while this one is written out
                if (j + 1 < n) query(qi + 1);
                sums[self] = l;
                if constexpr (kParted) maxima[self] = rounded;   // free until the next chunk's
                head_sync();
                const float total = __fadd_rn(__fadd_rn(sums[0], sums[64]), __fadd_rn(sums[128], sums[192]));
                float divisor = total;
                if constexpr (kParted)
                    divisor = __fadd_rn(__fadd_rn(maxima[0], maxima[64]), __fadd_rn(maxima[128], maxima[192]));
                // The last value product implies everything before it: each of its chunks passed
                // only arrivals of warps that had all they waited for.  A head's warps agree on
                // it, so that its row is written in full or not at all.  (The barrier also puts
                // the other lanes' accesses behind lane 0's wait, and the next segment's sums
                // behind the reads of these.)
                if (lane == 0) wait_quiet(smem_addr(&bars->stage_empty[j % kStages]), (j / kStages) & 1, ok);
                ok = !head_any(!ok);
                tc_fence_after_sync();
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, divisor);
                const bool whole = seg == 0 && ci + 1 == cut.per_query;
                const bool narrow = whole && (!kParted || p.wide == 0);
                const float lse2 =
                    total == 0.0f ? -INFINITY : __fadd_rn(__fsub_rn(m, kLift), log2f(total));
                // A piece that does not begin its query is its pair's first: slot 0.  Rows leave
                // through a part of the probabilities' buffers, free now, so that four lanes write
                // 64 bytes of one row: an eighth for each warp, in the rows of its own heads,
                // which their other warps do not write before it is done (head_any); those of
                // the other heads may be at the next query already.
                const int64_t slot = 2 * pair + (seg == 0 ? 1 : 0);
                float* const pieces = static_cast<float*>(p.workspace);
                const int64_t at = (whole ? qi : slot) * p.num_heads;
                const int64_t dst_row = narrow ? 1024 : 2048;
                uint8_t* const dst = (whole ? static_cast<uint8_t*>(p.out)
                                            : reinterpret_cast<uint8_t*>(pieces)) +
                                     at * dst_row + (2 * half + part) * (dst_row >> 2);
                const uint32_t st = smem_addr(smem + kOffP) + (warp >> 2) * kPBytes + (warp & 1) * (kPBytes / 2) +
                                    (warp >> 1 & 1) * (kPBytes / 4);
                const uint32_t mine = st + lane * 64 + (((lane >> 1) & 3) << 4);
                const int head0 = static_cast<int>(rank) * kPairHeads + (warp & 1) * 32;
                const int step = narrow ? 32 : 16;
#pragma unroll 1
                for (int c = 0; c < 128; c += step) {           // 64 bytes of each row
                    float t[16];
                    tmem_ld16(tmem + lanes + 128 * part + c, t);
                    if (narrow) {
                        sts16(mine, pack8(t, inv));
                        sts16(mine ^ 16u, pack8(t + 8, inv));
                        tmem_ld16(tmem + lanes + 128 * part + c + 16, t);
                        sts16(mine ^ 32u, pack8(t, inv));
                        sts16(mine ^ 48u, pack8(t + 8, inv));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sts16(mine ^ (i << 4),
                                  make_uint4(__float_as_uint(__fmul_rn(t[4 * i], inv)),
                                             __float_as_uint(__fmul_rn(t[4 * i + 1], inv)),
                                             __float_as_uint(__fmul_rn(t[4 * i + 2], inv)),
                                             __float_as_uint(__fmul_rn(t[4 * i + 3], inv))));
                    }
                    __syncwarp();
                    uint8_t* const to = dst + c * (narrow ? 2 : 4) + (lane & 3) * 16;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2);
                        const uint4 x = lds16_at(st + r * 64 + (((lane ^ (r >> 1)) & 3) << 4));
                        if (head0 + r < p.num_heads && ok) st16(to + (head0 + r) * dst_row, x);
                    }
                    __syncwarp();
                }
                if (half == 0 && part == 0 && head < p.num_heads) {
                    float* const to = whole ? p.lse : pieces + 2 * static_cast<int64_t>(cut.pairs) * p.num_heads * 512;
                    to[at + head] = !ok ? __uint_as_float(kUnwritten) : narrow ? __fmul_rn(lse2, kLn2) : lse2;
                }
                tc_fence_before_sync();
                m = -INFINITY;
                l = 0.0f;
                if constexpr (kParted) rounded = 0.0f;
                fresh = true;
                seg = 0;
            }
            if (++ci == cut.per_query) {
                ci = 0;
                ++qi;
            }
        }
        // after a wait that gave up, blocks of a query may still be on their way (otherwise this
        // thread has waited for all that it asked for)
        if (threadIdx.x == kPollThread && !ok) {
            if (bars->next_loads > 0) wait_landed(smem_addr(&bars->q_next), (bars->next_loads - 1) & 1);
            if (bars->live_loads > 0) wait_landed(smem_addr(&bars->q_live), (bars->live_loads - 1) & 1);
        }
        __syncwarp();
    }
    if (!ok) bars->timed_out = 1;
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && bars->timed_out != 0) report(p.err, kErrTimeout);
    cluster_sync();   // no CTA leaves while the other's products or arrivals reach it
    if (warp == kMmaWarp) {
        if (rank != 0) wait_landed(smem_addr(&bars->drained), 0);   // the last arrival from the other CTA
        __syncwarp();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// The queries that the cut runs through: query, its first pair and how many work on it.
constexpr int kMaxPairs = 128;
// Four groups from this many pieces of a query on: 32 pieces (a query, 128 heads) 14.2 us a call with
// one group, 13.2 with four; ten (8 queries, 32 heads) 25.2 and 22.9; two or three (128 queries,
// cut, 128 heads, 9600 blocks) 86 and 135.
constexpr int kManyPieces = 8;
struct Cuts {
    int32_t n;
    int32_t query[kMaxPairs - 1];
    int16_t first[kMaxPairs - 1], pairs[kMaxPairs - 1];
    // entry c: its query, first pair, pieces
    __device__ int find(int c, int64_t& q, int& g) const {
        q = query[c];
        g = first[c];
        return pairs[c];
    }
};
// The same of every query, where there are more pairs; those of one pair are whole.
struct ManyCuts {
    Cut cut;
    __device__ int find(int c, int64_t& q, int& g) const {
        q = c;
        const int64_t a = cut.pair_of(q * cut.per_query), z = cut.pair_of((q + 1) * cut.per_query - 1);
        g = static_cast<int>(a);
        return z > a ? static_cast<int>(z - a) + 1 : 0;
    }
};

// Joins the pieces of each cut query: out = sum_i exp2(lse_i - lse) rows_i.  A block takes one
// head of one query, four dims a thread; for many pieces, four groups of 128 threads take every
// fourth piece and add up in shared memory.  A few pieces are a matter of throughput, many of
// latency, so the first loads do not wait for the log-sum-exps.
constexpr int kJoinFirst = 4;
template <int kGroups, typename CutsOf>
__global__ void __launch_bounds__(128 * kGroups)
    join_kernel(const AttentionParams p, const int32_t pairs, const __grid_constant__ CutsOf cuts) {
    __shared__ float4 part[kGroups][kGroups > 1 ? 128 : 1];
    const int32_t c = blockIdx.x / p.num_heads;
    const int32_t head = blockIdx.x - c * p.num_heads;
    int64_t query;
    int g0;
    const int n = cuts.find(c, query, g0);
    const int d = threadIdx.x & 127, group = threadIdx.x >> 7;
    pdl_wait_previous();
    pdl_release_next();
    if (n == 0) return;
    const float* const rows = static_cast<const float*>(p.workspace);
    const float* const lses = rows + 2 * static_cast<int64_t>(pairs) * p.num_heads * 512 + head;
    // the first piece ends its pair's run (slot 1), the others begin theirs (slot 0)
    auto slot = [&](int i) -> int32_t { return (2 * (g0 + i) + (i == 0 ? 1 : 0)) * p.num_heads; };
    auto load = [&](int i) -> float4 {
        return *reinterpret_cast<const float4*>(rows + (static_cast<int64_t>(slot(i)) + head) * 512 + 4 * d);
    };
    // this thread's first pieces are on their way while the log-sum-exps are read
    float4 first[kJoinFirst];
#pragma unroll
    for (int u = 0; u < kJoinFirst; ++u) {
        const int i = group + u * kGroups;
        first[u] = i < n ? load(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    // the pieces' log-sum-exps, one a lane
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    bool unwritten = false;
    for (int i = lane; i < n; i += 32) {
        const float x = lses[slot(i)];
        unwritten |= is_unwritten(x);
        m = fmaxf(m, x);
    }
    unwritten = __any_sync(kFull, unwritten) != 0;   // the same in every warp
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
    const float ref = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
    for (int i = lane; i < n; i += 32) sum = __fadd_rn(sum, exp2_approx(__fsub_rn(lses[slot(i)], ref)));
    sum = warp_sum(sum);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](int i, const float4& t) {
        const float w = exp2_approx(__fsub_rn(lses[slot(i)], ref));
        acc.x = __fmaf_rn(w, t.x, acc.x);
        acc.y = __fmaf_rn(w, t.y, acc.y);
        acc.z = __fmaf_rn(w, t.z, acc.z);
        acc.w = __fmaf_rn(w, t.w, acc.w);
    };
#pragma unroll
    for (int u = 0; u < kJoinFirst; ++u)
        if (group + u * kGroups < n) add(group + u * kGroups, first[u]);
#pragma unroll 4
    for (int i = group + kJoinFirst * kGroups; i < n; i += kGroups) add(i, load(i));
    if constexpr (kGroups > 1) {
        part[group][d] = acc;
        __syncthreads();
        if (group != 0) return;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) {
            const float4 t = part[i][d];
            acc.x = __fadd_rn(acc.x, t.x);
            acc.y = __fadd_rn(acc.y, t.y);
            acc.z = __fadd_rn(acc.z, t.z);
            acc.w = __fadd_rn(acc.w, t.w);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    const float lse2 = sum == 0.0f ? -INFINITY : __fadd_rn(m, log2f(sum));
    const uint2 v = make_uint2(pack_bf16x2_rn(__fmul_rn(acc.x, inv), __fmul_rn(acc.y, inv)),
                               pack_bf16x2_rn(__fmul_rn(acc.z, inv), __fmul_rn(acc.w, inv)));
    const int64_t at = query * p.num_heads + head;
    if (unwritten) {
        if (threadIdx.x == 0) p.lse[at] = __uint_as_float(kUnwritten);
        return;
    }
    if (p.wide != 0) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * 512 + 4 * d) =
            make_float4(__fmul_rn(acc.x, inv), __fmul_rn(acc.y, inv), __fmul_rn(acc.z, inv), __fmul_rn(acc.w, inv));
        if (threadIdx.x == 0) p.lse[at] = lse2;
        return;
    }
    st8(static_cast<uint8_t*>(p.out) + at * 1024 + 8 * d, v);
    if (threadIdx.x == 0) p.lse[at] = __fmul_rn(lse2, kLn2);
}

// ---------------------------------------------------------------- weights
//
// weights[i, k] += sum over h of exp(s[i, h, k] - lse[i, h]): the logits once more, now that
// every head's lse is known (keeping them would take num_heads * 4 bytes an entry, 64 times
// what the record has).  Here the records are the rows of the product (M = 128) and the heads
// its columns, so a thread has all heads of one record and sums them in its registers, in the
// heads' order.  One CTA an SM; a tile is 128 records of one query.
//   * four warps fetch indices, scale rows and, a quarter-row (64 bytes) at a time, the codes;
//   * 16 warps dequantise 64 dims of the tile at a time (16 KB a stage), eight warps each stage;
//   * one thread multiplies them by the query's heads, which lie in shared memory, into one of
//     two accumulators;
//   * four warps turn the accumulator into the records' sums and add them to the weights.
// Measured at 64 queries of 128 heads and 2049 entries: 30 us, against 45 us with one group of
// 16 warps a stage, one stage less and whole half-rows.  The products alone are 17 GFLOP
// (9 us); what is left is the dequantisation's instructions and the latencies between a stage's
// filling, its product and its next filling: two or three stages are all that shared memory
// holds beside 128 heads.

constexpr int kTileKeys = 128;
constexpr int kWSoftWarps = 4;                              // warp w: tensor-memory lanes 32w ..
constexpr int kWDequantWarps = 16;
constexpr int kWMmaWarp = kWSoftWarps + kWDequantWarps;
constexpr int kWGatherWarps = 4;
constexpr int kWFirstGather = kWMmaWarp + 1;
constexpr int kWeightThreads = (kWFirstGather + kWGatherWarps) * 32;
constexpr int kWGroups = 2;                                 // of dequantisation warps
constexpr int kWGroupWarps = kWDequantWarps / kWGroups;
constexpr int kWIndexRing = 4, kWIndexAhead = 3;            // tiles of indices
constexpr uint32_t kWStageBytes = kTileKeys * kRowBytes;    // 64 dims of a tile
constexpr uint32_t kWRawBytes = kTileKeys * 64;             // quarter-rows of a tile: 128 dims

// Shared memory for queries of up to kHeads heads: the query, stages, quarter-rows in flight,
// scales, heads' lse, indices, live bits, barriers.
template <int kHeads>
struct WeightSmem {
    static constexpr int kStages = kHeads <= 64 ? 4 : 3;
    static constexpr int kRaw = kHeads <= 64 ? 8 : 5;
    struct alignas(8) Barriers {
        uint64_t q_full, q_free;               // the query is in place; its last product is done
        uint64_t raw[kRaw], raw_empty[kRaw];   // quarter-rows landed (the first with the scales); read
        uint64_t scales_empty[2];              // a tile's scales are read
        uint64_t a_full[kStages], a_empty[kStages];
        uint64_t acc_full[2], acc_empty[2];
        uint64_t drained;                      // every product that was issued is complete
        uint32_t tmem_base;
        int32_t timed_out;
    };
    static constexpr uint32_t kStagesAt = kHeads * 1024;
    static constexpr uint32_t kRawAt = kStagesAt + kStages * kWStageBytes;
    static constexpr uint32_t kScalesAt = kRawAt + kRaw * kWRawBytes;          // [2 tiles][128][16]
    static constexpr uint32_t kLseAt = kScalesAt + 2 * kTileKeys * 16;         // [kHeads] lse in powers of two
    static constexpr uint32_t kIndexAt = kLseAt + kHeads * 4;                  // [kWIndexRing][128]
    static constexpr uint32_t kLiveAt = kIndexAt + kWIndexRing * kTileKeys * 4;   // [8][4] bits
    static constexpr uint32_t kBarsAt = kLiveAt + 8 * 16;
    static constexpr size_t kBytes = 1024 + kBarsAt + sizeof(Barriers);
    static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
};

template <int kHeads>
__global__ void __launch_bounds__(kWeightThreads, 1)
    weight_kernel(const AttentionParams p, const int64_t tiles, const int32_t n_pad,
                  const __grid_constant__ CUtensorMap q_map) {
    using M = WeightSmem<kHeads>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    typename M::Barriers* const bars = reinterpret_cast<typename M::Barriers*>(smem + M::kBarsAt);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // tiles i0 .. i0 + n - 1 of all queries' tiles, one query after another
    const int64_t total = p.num_queries * tiles;
    const int64_t i0 = total * blockIdx.x / gridDim.x;
    const int n = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x - i0);

    if (warp == kWMmaWarp) {
        tmem_alloc(smem_addr(&bars->tmem_base), 256);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&bars->q_full), 1);
        mbar_init(smem_addr(&bars->q_free), 1);
        mbar_init(smem_addr(&bars->drained), 1);
        for (int s = 0; s < M::kRaw; ++s) {
            mbar_init(smem_addr(&bars->raw[s]), kWGatherWarps * (1 + 32));
            mbar_init(smem_addr(&bars->raw_empty[s]), kWDequantWarps);
        }
        for (int s = 0; s < M::kStages; ++s) {
            mbar_init(smem_addr(&bars->a_full[s]), kWGroupWarps);
            mbar_init(smem_addr(&bars->a_empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&bars->scales_empty[s]), kWDequantWarps);
            mbar_init(smem_addr(&bars->acc_full[s]), 1);
            mbar_init(smem_addr(&bars->acc_empty[s]), kWSoftWarps);
        }
        bars->timed_out = 0;
        mbar_init_fence();
    }
    pdl_wait_previous();
    pdl_release_next();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    bool ok = true;
    int64_t qi = i0 / tiles;
    int64_t ti = i0 - qi * tiles;

    if (warp >= kWSoftWarps && warp < kWMmaWarp) {
        // ------------------------------------------------------------- dequantisation
        // Eight warps fill every other stage, eight the ones between, so that one group's loads,
        // stores and waits lie behind the other's arithmetic.  A warp takes 16 records, a lane
        // 32 dims of one: one scale and one 16-byte read.
        const int w = warp - kWSoftWarps;
        const int group = w / kWGroupWarps;
        const int r = (w % kWGroupWarps) * 16 + (lane & 7) + 8 * (lane >> 4);
        const int v = (lane >> 3) & 1;
        const uint32_t raw0 = smem_addr(smem + M::kRawAt) + r * 64 + (((2 * group + v) ^ (r >> 1 & 3)) << 4);
        const uint32_t scale0 = smem_addr(smem + M::kScalesAt) + r * 16 + 2 * group + v;
        const uint32_t dst0 = smem_addr(smem + M::kStagesAt) + r * kRowBytes;
        Ring<M::kRaw> rw;
        int stage = group;                 // every other one of the ring's
        uint32_t turn = 0;                 // of the ring
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {   // 128 dims: 64 for each group
                // every warp waits for itself: at a barrier of the warps each stage took as long
                // as the slowest of them
                if (!warp_wait(smem_addr(&bars->raw[rw.s]), rw.parity, ok)) break;
                if (turn > 0 && !warp_wait(smem_addr(&bars->a_empty[stage]), (turn - 1) & 1, ok)) break;
                const uint4 codes = lds16_at(raw0 + rw.s * kWRawBytes);
                uint32_t s;
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s)
                             : "r"(scale0 + (j & 1) * kTileKeys * 16 + 4 * h) : "memory");
                const uint32_t f = e2m1_factor(s), dst = dst0 + stage * kWStageBytes;
                sts16(dst + (((4 * v + 0) ^ (r & 7)) << 4), dequant8_e2m1(codes.x, f));
                sts16(dst + (((4 * v + 1) ^ (r & 7)) << 4), dequant8_e2m1(codes.y, f));
                sts16(dst + (((4 * v + 2) ^ (r & 7)) << 4), dequant8_e2m1(codes.z, f));
                sts16(dst + (((4 * v + 3) ^ (r & 7)) << 4), dequant8_e2m1(codes.w, f));
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&bars->raw_empty[rw.s]));
                    if (h == 3) mbar_arrive(smem_addr(&bars->scales_empty[j & 1]));
                    mbar_arrive(smem_addr(&bars->a_full[stage]));
                }
                rw.next();
                stage += kWGroups;
                if (stage >= M::kStages) {
                    stage -= M::kStages;
                    ++turn;
                }
            }
        }
    } else if (warp >= kWFirstGather) {
        // ------------------------------------------------------------- raw records
        // A warp has 32 records of the tile: a lane finds one's row, four lanes copy a
        // quarter-row.  Four warps: one alone took 110 cycles a copy instruction, 1800 a quarter
        // of the tile, which then set the pace.
        const int rec = (warp - kWFirstGather) * 32;
        const uint32_t ring = smem_addr(smem + M::kIndexAt) + 4 * (rec + lane);
        int ahead = 0;
        auto fetch = [&]() {
            if (ahead < n) {
                const uint32_t to = ring + (ahead % kWIndexRing) * kTileKeys * 4;
                const int64_t k = ti * kTileKeys + rec + lane;
                if (k < p.topk) cp_async4(to, p.indices + qi * p.index_stride + k);
                else asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(-1) : "memory");
                if (++ti == tiles) {
                    ti = 0;
                    ++qi;
                }
                ++ahead;
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kWIndexAhead; ++i) fetch();
        const int c = lane & 3;   // 16-byte chunk of the quarter-row
        const uint32_t to0 = smem_addr(smem + M::kRawAt) + (rec + (lane >> 2)) * 64 + ((c ^ (lane >> 3 & 3)) << 4);
        Ring<M::kRaw> rw;
        int quarters = 0;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
            cp_async_wait<kWIndexAhead - 1>();
            int32_t slot;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(slot)
                         : "r"(ring + (j % kWIndexRing) * kTileKeys * 4) : "memory");
            const bool is = slot >= 0 && slot < p.num_slots;
            const uint32_t live = __ballot_sync(kFull, is);
            uint32_t page, row;
            page_row(is ? static_cast<uint32_t>(slot) : 0u, static_cast<uint32_t>(p.block_size), page, row);
            const int64_t at = static_cast<int64_t>(page) * p.page_stride;
            const int32_t rows = static_cast<int32_t>(at >> 8) + static_cast<int32_t>(row);   // of 256 bytes
            const uint8_t* const scales = p.cache + at + static_cast<int64_t>(p.block_size) * 256 + row * 16u;
            const uint8_t* from[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                from[i] = p.cache + 16 * c +
                          static_cast<int64_t>(__shfl_sync(kFull, rows, 8 * i + (lane >> 2))) * 256;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                if (quarters >= M::kRaw && !warp_wait(smem_addr(&bars->raw_empty[rw.s]), rw.parity ^ 1u, ok)) break;
                if (h == 0) {
                    if (j >= 2 && !warp_wait(smem_addr(&bars->scales_empty[j & 1]), ((j >> 1) - 1) & 1, ok)) break;
                    cp_async16_or_zeros(smem_addr(smem + M::kScalesAt) + ((j & 1) * kTileKeys + rec + lane) * 16,
                                        scales, is);
                    if (lane == 0)
                        *reinterpret_cast<uint32_t*>(smem + M::kLiveAt + (j & 7) * 16 + rec / 8) = live;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    cp_async16_or_zeros(to0 + rw.s * kWRawBytes + i * 512, from[i] + 64 * h,
                                        (live >> (8 * i + (lane >> 2)) & 1u) != 0u);
                const uint32_t bar = smem_addr(&bars->raw[rw.s]);
                cp_async_arrive(bar);
                if (lane == 0) mbar_arrive(bar);
                rw.next();
                ++quarters;
            }
            fetch();
        }
        cp_async_wait<0>();   // the copies in flight land before the CTA leaves
    } else if (warp == kWMmaWarp) {
        // ------------------------------------------------------------- products
        const uint32_t elected = elect_lane();
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n_pad >> 3) << 17) |
                               (static_cast<uint32_t>(128 >> 4) << 24);
        const uint64_t a_desc = sw128_desc(smem_addr(smem + M::kStagesAt));
        const uint64_t q_desc = sw128_desc(smem_addr(smem));
        const uint32_t a_lo = static_cast<uint32_t>(a_desc), q_lo = static_cast<uint32_t>(q_desc);
        const uint32_t q_block = static_cast<uint32_t>(n_pad) * kRowBytes;   // 64 dims of the query
        Ring<M::kStages> st;
        uint32_t loads = 0;   // of queries, issued
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            if (j == 0 || ti == 0) {   // the next query, once the last product of the one before is done
                if (j > 0 && !warp_wait(smem_addr(&bars->q_free), (loads - 1) & 1, ok)) break;
                if (elected) {
                    mbar_expect_tx(smem_addr(&bars->q_full), 8 * q_block);
#pragma unroll 1
                    for (int b = 0; b < 8; ++b)
                        tma_load_3d(smem_addr(smem) + b * q_block, &q_map, smem_addr(&bars->q_full), 64 * b, 0,
                                    static_cast<int32_t>(qi));
                }
                ++loads;
                if (!warp_wait(smem_addr(&bars->q_full), (loads - 1) & 1, ok)) break;
            }
            if (j >= 2 && !warp_wait(smem_addr(&bars->acc_empty[j & 1]), ((j >> 1) - 1) & 1, ok)) break;
#pragma unroll 1
            for (int h = 0; h < 8; ++h) {
                if (!warp_wait(smem_addr(&bars->a_full[st.s]), st.parity, ok)) break;
                tc_fence_after_sync();
                if (elected) {
                    const uint32_t a = a_lo + st.s * (kWStageBytes >> 4);
                    const uint32_t q = q_lo + ((h * q_block) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ss(tmem + 128 * (j & 1), desc_at(a_desc, a + 2 * k), desc_at(q_desc, q + 2 * k),
                                    idesc, h != 0 || k != 0);
                    mma_commit(smem_addr(&bars->a_empty[st.s]));
                }
                __syncwarp();
                st.next();
            }
            if (!ok) break;
            if (elected) mma_commit(smem_addr(&bars->acc_full[j & 1]));
            if (++ti == tiles) {
                ti = 0;
                ++qi;
                if (elected && j + 1 < n) mma_commit(smem_addr(&bars->q_free));
            }
            __syncwarp();
        }
        // whatever ended the loop, no product and no block of a query is under way when the CTA leaves
        if (elected) mma_commit(smem_addr(&bars->drained));
        __syncwarp();
        if (!wait_landed(smem_addr(&bars->drained), 0)) ok = false;
        if (loads > 0 && !wait_landed(smem_addr(&bars->q_full), (loads - 1) & 1)) ok = false;
        __syncwarp();
    } else {
        // ------------------------------------------------------------- sums
        float* const lse = reinterpret_cast<float*>(smem + M::kLseAt);
        const float scale = __fmul_rn(p.sm_scale, kLog2e);
        const uint64_t scale2 = f32x2(scale, scale);
        const int key = warp * 32 + lane;
        bool known = false;                                  // every head's lse of this query is
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            if (j == 0 || ti == 0) {
                group_sync(kSoftmaxBar, kWSoftWarps * 32);   // the query before is read
                const int h = threadIdx.x;                   // 0 .. 127
                bool unwritten = false;
                if (h < kHeads) {
                    const float x = h < p.num_heads ? p.lse[qi * p.num_heads + h] : INFINITY;
                    unwritten = is_unwritten(x);
                    lse[h] = __fmul_rn(-kLog2e, x);          // no head: exp2(-inf) = 0
                }
                known = !group_any(kSoftmaxBar, kWSoftWarps * 32, unwritten);
            }
            if (ok) warp_wait(smem_addr(&bars->acc_full[j & 1]), (j >> 1) & 1, ok);
            tc_fence_after_sync();
            const uint32_t bits = *reinterpret_cast<const uint32_t*>(smem + M::kLiveAt + (j & 7) * 16 + 4 * warp);
            const bool live = (bits >> lane & 1u) != 0u;
            uint64_t sum2 = f32x2(0.0f, 0.0f);
#pragma unroll 1
            for (int c = 0; c < n_pad; c += 16) {
                float v[16];
                tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 128 * (j & 1) + c, v);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(lse + c + i);
                    float a, b;
                    f32x2_split(fma_f32x2(f32x2(v[i], v[i + 1]), scale2, f32x2(m.x, m.y)), a, b);
                    sum2 = add_f32x2(sum2, f32x2(exp2_flush(a), exp2_flush(b)));
                    f32x2_split(fma_f32x2(f32x2(v[i + 2], v[i + 3]), scale2, f32x2(m.z, m.w)), a, b);
                    sum2 = add_f32x2(sum2, f32x2(exp2_flush(a), exp2_flush(b)));
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(smem_addr(&bars->acc_empty[j & 1]));
            if (live && ok && known) {
                float even, odd;
                f32x2_split(sum2, even, odd);
                float* const dst = p.weights + qi * p.weight_stride + ti * kTileKeys + key;
                *dst = __fadd_rn(*dst, __fadd_rn(even, odd));
            }
            if (++ti == tiles) {
                ti = 0;
                ++qi;
            }
        }
    }
    if (!ok) atomicOr(&bars->timed_out, 1);
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && bars->timed_out != 0) report(p.err, kErrTimeout);
    if (warp == kWMmaWarp) tmem_dealloc(tmem, 256);
}

cudaError_t make_cut(int64_t num_queries, int64_t topk, int32_t num_heads, Cut* cut) {
    int32_t pairs = 0;
    const cudaError_t e = resident_pairs(reinterpret_cast<const void*>(attend_kernel<false>), kAttendThreads, kAttendSmem, &pairs);
    if (e != cudaSuccess) return e;
    cut->per_query = topk == 0 ? 1 : (topk + kChunkKeys - 1) / kChunkKeys;
    cut->total = num_queries * cut->per_query;
    if (pairs > kMaxPairs) pairs = kMaxPairs;
    cut->pairs = static_cast<int32_t>(cut->total < pairs ? cut->total : pairs);
    cut->each = 0;
    // Whole queries, as many for each pair, where the longest run is then no longer than the even
    // cut's and what the pieces' fp32 rows and the kernel that joins them cost, in chunks of 1 us:
    // five, and one for 9 heads where every pair writes two pieces; fewer pieces cost less.
    // Measured, us in a graph whole and cut: 128 queries x 2048 entries x 128 heads (64 chunks,
    // 54) 75 and 86; 120 x 1088 x 128 (34, 27) 45 and 57; 90 x 1600 (50, 30) x 128 heads 60.4 and
    // 60.0, x 64 60 and 53, x 16 59 and 46; 100 x 1024 (32, 22) x 64 42 and 44, x 32 41 and 39;
    // 40 x 640 x 16 (10, 6) 16 and 20; 37 x 1531 x 16 (24, 12) 30 and 25.5.  Few queries: 1 x 1280 x
    // 128 (20, 1) 26.0 and 12.5; 1 x 256 x 128 (4, 1) 10.0 and 10.8; 4 x 512 x 128 (8, 1) 14.5 and
    // 14.2; 16 x 1280 x 128 (20, 5) 26.7 and 23.6; 32 x 1280 x 128 (20, 9) 26.9 and 29.5; 2 x 512 x 32
    // (8, 1) 13.9 and 10.3.  Of 420 sizes of 1 .. 160 queries, 8 .. 128 heads and 128 .. 2048
    // entries the slower form is taken in four, by 6 to 9 %.
    const int64_t each = (num_queries + pairs - 1) / pairs;
    const int64_t pieces = cut->pairs + (cut->total > pairs ? (num_queries < pairs ? num_queries : pairs) : 0);
    if (each * cut->per_query <= (cut->total + pairs - 1) / pairs + 5 + num_heads * pieces / (18 * pairs)) {
        cut->each = each;
        cut->pairs = static_cast<int32_t>((num_queries + each - 1) / each);
    }
    const int64_t run = cut->each > 0 ? cut->each * cut->per_query : (cut->total + pairs - 1) / pairs;
    if (cut->per_query > kRunChunks && run > kRunChunks) {
        cut->each = 0;
        cut->pairs = static_cast<int32_t>(pairs * ((cut->total + pairs * kRunChunks - 1) / (pairs * kRunChunks)));
    }
    return cudaSuccess;
}

// Whether some query is cut, so that there are pieces to join.
bool has_pieces(const Cut& cut) {
    for (int32_t g = 1; g < cut.pairs; ++g)
        if (cut.begin(g) % cut.per_query != 0) return true;
    return false;
}

// The queries that pairs' runs begin inside of.
int find_cuts(const Cut& cut, Cuts* cuts) {   // returns the most pieces of a query
    cuts->n = 0;
    int most = 0;
    for (int32_t g = 1; g < cut.pairs; ++g) {
        const int64_t begin = cut.begin(g), q = begin / cut.per_query;
        if (begin - q * cut.per_query == 0) continue;
        if (cuts->n == 0 || cuts->query[cuts->n - 1] != q) {
            cuts->query[cuts->n] = static_cast<int32_t>(q);
            cuts->first[cuts->n] = static_cast<int16_t>(g - 1);
            cuts->pairs[cuts->n++] = 1;
        }
        if (++cuts->pairs[cuts->n - 1] > most) most = cuts->pairs[cuts->n - 1];
    }
    return most;
}

// The queries [num_queries, num_heads, 512] as a 3-D tensor map with boxes of 64 dims x `heads`
// heads and the 128-byte swizzle; heads past num_heads read as zeros.
cudaError_t q_tensor_map(const AttentionParams& p, int heads, CUtensorMap* map) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {512, static_cast<cuuint64_t>(p.num_heads),
                                static_cast<cuuint64_t>(p.num_queries)};
    const cuuint64_t strides[2] = {1024, static_cast<cuuint64_t>(1024) * p.num_heads};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), 1};
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
    const cudaError_t e = make_cut(num_queries, topk, num_heads, &cut);
    if (e != cudaSuccess) return e;
    // two pieces a pair: a row and a log-sum-exp for each head
    *bytes = has_pieces(cut) ? 2 * static_cast<int64_t>(cut.pairs) * num_heads * (512 + 1) * 4 : 0;
    return cudaSuccess;
}

cudaError_t launch_sparse_attention(const AttentionParams& p, cudaStream_t stream) {
    Cut cut;
    cudaError_t e = make_cut(p.num_queries, p.topk, p.num_heads, &cut);
    if (e != cudaSuccess) return e;
    CUtensorMap q_map;
    e = q_tensor_map(p, kPairHeads, &q_map);
    if (e != cudaSuccess) return e;
    const bool parted = p.parted != 0;
    if (parted) {   // the kernel's limit of shared memory is set with this
        int32_t pairs = 0;
        e = resident_pairs(reinterpret_cast<const void*>(attend_kernel<true>), kAttendThreads, kAttendSmem, &pairs);
        if (e != cudaSuccess) return e;
    }
    e = launch_kernel(parted ? attend_kernel<true> : attend_kernel<false>, 2 * static_cast<int64_t>(cut.pairs),
                      kAttendThreads, kAttendSmem, stream, p.pdl, p, cut, q_map);
    if (e != cudaSuccess) return e;
    if (cut.pairs > kMaxPairs) {
        const ManyCuts cuts = {cut};
        e = launch_kernel(join_kernel<4, ManyCuts>, p.num_queries * p.num_heads, 512, 0, stream, p.pdl, p, cut.pairs, cuts);
        if (e != cudaSuccess) return e;
    } else {
        Cuts cuts;
        const int most = find_cuts(cut, &cuts);
        if (cuts.n > 0) {
            const int64_t blocks = static_cast<int64_t>(cuts.n) * p.num_heads;
            e = most >= kManyPieces ? launch_kernel(join_kernel<4, Cuts>, blocks, 512, 0, stream, p.pdl, p, cut.pairs, cuts)
                                    : launch_kernel(join_kernel<1, Cuts>, blocks, 128, 0, stream, p.pdl, p, cut.pairs, cuts);
            if (e != cudaSuccess) return e;
        }
    }
    if (p.weights == nullptr || p.topk == 0) return e;
    const int n_pad = (p.num_heads + 15) / 16 * 16;   // columns of the product
    e = q_tensor_map(p, n_pad, &q_map);
    if (e != cudaSuccess) return e;
    const auto kernel = p.num_heads <= 64 ? weight_kernel<64> : weight_kernel<128>;
    const size_t smem = p.num_heads <= 64 ? WeightSmem<64>::kBytes : WeightSmem<128>::kBytes;
    int64_t warps = 0;
    e = resident_warps(reinterpret_cast<const void*>(kernel), kWeightThreads, smem, &warps);
    if (e != cudaSuccess) return e;
    const int64_t ctas = warps / (kWeightThreads / 32);
    const int64_t tiles = (p.topk + kTileKeys - 1) / kTileKeys;
    const int64_t blocks = p.num_queries * tiles < ctas ? p.num_queries * tiles : ctas;
    return launch_kernel(kernel, blocks, kWeightThreads, smem, stream, p.pdl, p, tiles, n_pad, q_map);
}

}  // namespace gkr
