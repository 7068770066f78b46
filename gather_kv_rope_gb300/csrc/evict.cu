// Eviction from a cache by accumulated attention weight.
//
// Operation, per row (one sequence's list of records): entry p holds the slot indices[p]
// (negative: empty) and weights[p], the attention the record has received.  The last
// `recent` live entries are kept; of the others, those of the largest weights, the first
// entry where weights tie, until `keep` are kept in all.  The kept slots and weights leave
// in the row's order, so do the other live slots (the evicted ones).  A NaN weight ranks below
// every number, -0 with 0.
//
// The weight of the last entry to be kept is found by its bits: a weight's 32 bits map to an
// unsigned key in the order of the values, and four passes over the row, each counting the
// keys that share the bits found so far by their next 8 bits, fix one byte of it each.  A
// last pass over the row in order then knows each entry's fate -- kept if newer, or above
// that key, or equal to it and among the first `ties` such -- and its place, from running
// counts.  Counts are whole numbers, so the result does not depend on the order of threads.
#include "device.cuh"
#include "launch.h"

namespace gkr {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;

// A weight's key: unsigned order = order of the values; NaN 0 (below -inf), -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(__fadd_rn(w, 0.0f));
    return (b & 0x80000000u) != 0u ? ~b : (b | 0x80000000u);
}

// The block's sum of v, in every thread.
__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t* shared, int warp, int lane) {
    v = __reduce_add_sync(kFull, v);
    __syncthreads();   // the last use of `shared` is over
    if (lane == 0) shared[warp] = v;
    __syncthreads();
    return __reduce_add_sync(kFull, lane < kEvictWarps ? shared[lane] : 0);
}

// Exclusive prefix of v over the block's threads; *total = the sum.
__device__ __forceinline__ int32_t block_prefix(int32_t v, int32_t* shared, int warp, int lane,
                                                int32_t* total) {
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) shared[warp] = x;
    __syncthreads();
    const int32_t w = shared[lane];   // kEvictWarps == 32
    *total = __reduce_add_sync(kFull, w);
    return x - v + __reduce_add_sync(kFull, lane < warp ? w : 0);
}

__global__ void __launch_bounds__(kEvictThreads, 1) evict_kernel(const EvictParams p) {
    static_assert(kEvictWarps == 32, "block_prefix");
    __shared__ int32_t shared[kEvictWarps];
    __shared__ int32_t hist[256];
    __shared__ int32_t found[2];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x;
    const int32_t L = p.length;
    pdl_wait_previous();
    pdl_release_next();
    const int32_t* const idx = p.indices + r * p.index_stride;
    const float* const wts = p.weights + r * p.weight_stride;

    int32_t live = 0;
    for (int32_t i = threadIdx.x; i < L; i += kEvictThreads) live += idx[i] >= 0 ? 1 : 0;
    live = block_sum(live, shared, warp, lane);
    const int32_t fresh = p.recent < live ? p.recent : live;   // protected entries
    const int32_t old = live - fresh;                          // the first `old` live ones compete
    int32_t room = p.keep - fresh < old ? p.keep - fresh : old;

    // the key of the last old entry kept, and how many of its equals stay
    uint32_t key = 0;
    int32_t ties = old;
    if (room < old) {
        uint32_t mask = 0;
        ties = room;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            int32_t before = 0;
            for (int32_t base = 0; base < L; base += kEvictThreads) {
                const int32_t i = base + threadIdx.x;
                const bool is = i < L && idx[i] >= 0;
                int32_t n;
                const int32_t rank = before + block_prefix(is ? 1 : 0, shared, warp, lane, &n);
                before += n;
                if (is && rank < old) {
                    const uint32_t k = weight_key(wts[i]);
                    if ((k & mask) == (key & mask)) atomicAdd(&hist[(k >> shift) & 255u], 1);
                }
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                int32_t left = ties;
                int d = 255;
                while (d > 0 && hist[d] < left) left -= hist[d--];
                found[0] = d;
                found[1] = left;
            }
            __syncthreads();
            key |= static_cast<uint32_t>(found[0]) << shift;
            mask |= 255u << shift;
            ties = found[1];
            __syncthreads();
        }
    }
    int32_t seen = 0, tied = 0, kept = 0, gone = 0;
    for (int32_t base = 0; base < L; base += kEvictThreads) {
        const int32_t i = base + threadIdx.x;
        const int32_t s = i < L ? idx[i] : -1;
        int32_t n;
        const int32_t rank = seen + block_prefix(s >= 0 ? 1 : 0, shared, warp, lane, &n);
        seen += n;
        const float w = s >= 0 ? wts[i] : 0.0f;
        const uint32_t k = weight_key(w);
        const bool competes = s >= 0 && rank < old;
        const bool equal = competes && k == key;
        const int32_t t = tied + block_prefix(equal ? 1 : 0, shared, warp, lane, &n);
        tied += n;
        const bool stays = s >= 0 && (!competes || room == old || k > key || (equal && t < ties));
        const bool goes = s >= 0 && !stays;
        const int32_t a = kept + block_prefix(stays ? 1 : 0, shared, warp, lane, &n);
        kept += n;
        const int32_t b = gone + block_prefix(goes ? 1 : 0, shared, warp, lane, &n);
        gone += n;
        if (stays) {
            p.kept[r * p.keep + a] = s;
            p.kept_weights[r * p.keep + a] = w;
        }
        if (goes) p.evicted[r * (L - p.keep) + b] = s;
    }
    for (int32_t i = kept + threadIdx.x; i < p.keep; i += kEvictThreads) {
        p.kept[r * p.keep + i] = -1;
        p.kept_weights[r * p.keep + i] = 0.0f;
    }
    for (int32_t i = gone + threadIdx.x; i < L - p.keep; i += kEvictThreads)
        p.evicted[r * (L - p.keep) + i] = -1;
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    return launch_kernel(evict_kernel, p.rows, kEvictThreads, 0, stream, p.pdl, p);
}

}  // namespace gkr
