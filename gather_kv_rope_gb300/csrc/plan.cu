// A step's plan on the GPU, from the lengths of the batch's requests: the pages that each
// request takes from the free list, the slot and position of every new token (what kv_insert
// takes), and the slots of what the requests hold (what sparse_attention and kv_gather take).
//
// With past_b and added_b tokens of request b, bs slots a page and W columns of the table:
//   held_b = min(ceil(past_b / bs), W), end_b = min(ceil((past_b + added_b) / bs), W),
//   take_b = end_b - held_b, offset_b = sum of take_c over c < b, starts_b = sum of added_c;
//   table[b, held_b + j] = free[offset_b + j] for j < take_b;
//   token i of request b is row starts_b + i: position past_b + i, slot
//   table[b, position / bs] * bs + position % bs.
//
// The outputs are a few bytes a token, so a launch's latency bounds all but the largest calls,
// and one launch does everything: every block sums the lengths of all requests for itself (a
// few KB from L2) and then finds the request of each of its rows by bisection in shared
// memory.  New pages are read from the free list, not from the table that other blocks are
// writing.  No atomics but for the error bits: the same call gives the same bytes.
#include "device.cuh"
#include "launch.h"

namespace gkr {

namespace {

constexpr int32_t kErrSlot = 1, kErrPos = 2, kErrIndex = 4;
constexpr int kPlanThreads = 512;
constexpr int64_t kIntMax = INT64_C(0x7FFFFFFF);

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(kFull, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Exclusive sums of f(0) .. f(n - 1), each at most kIntMax, into out[0 .. n] (clamped to
// kIntMax: `over` tells).  Each thread sums a run of consecutive elements.
template <typename F>
__device__ void block_sums(int n, int32_t* out, int64_t* scratch, bool& over, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int run = (n + kPlanThreads - 1) / kPlanThreads;
    const int first = min(n, static_cast<int>(threadIdx.x) * run), last = min(n, first + run);
    int64_t sum = 0;
    for (int i = first; i < last; ++i) sum += f(i);
    const int64_t upto = warp_inclusive(sum, lane);
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        const int64_t s = lane < kPlanThreads / 32 ? scratch[lane] : 0;
        const int64_t t = warp_inclusive(s, lane);
        if (lane < kPlanThreads / 32) scratch[lane] = t - s;
    }
    __syncthreads();
    int64_t at = scratch[warp] + upto - sum;
    for (int i = first; i < last; ++i) {
        out[i] = static_cast<int32_t>(min(at, kIntMax));
        at += f(i);
    }
    if (last == n && (first < n || threadIdx.x == 0)) {   // the thread of the last element
        out[n] = static_cast<int32_t>(min(at, kIntMax));
        over = at > kIntMax;
    }
    __syncthreads();
}

// The request b < n with sums[b] <= row < sums[b + 1]; row < sums[n].
__device__ __forceinline__ int find(const int32_t* sums, int n, int32_t row) {
    int lo = 0, hi = n;                     // sums[lo] <= row < sums[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct Split {   // x / bs by a shift where bs is a power of two
    uint32_t bs;
    int shift;   // or -1
    __device__ explicit Split(int32_t block_size) {
        bs = static_cast<uint32_t>(block_size);
        shift = (bs & (bs - 1u)) == 0u ? __ffs(block_size) - 1 : -1;
    }
    __device__ uint32_t page(uint32_t x) const { return shift >= 0 ? x >> shift : x / bs; }
    __device__ int64_t pages(int64_t x) const {   // ceil(x / bs), 0 <= x < 2^32
        const uint64_t y = static_cast<uint64_t>(x) + bs - 1u;
        if (shift >= 0) return static_cast<int64_t>(y >> shift);
        return static_cast<int64_t>(y <= 0xFFFFFFFFu ? static_cast<uint32_t>(y) / bs : y / bs);
    }
};

__global__ void __launch_bounds__(kPlanThreads) allocate_kernel(const AllocateParams p) {
    extern __shared__ int32_t sums[];       // starts[n + 1], offsets[n + 1]
    __shared__ int64_t scratch[kPlanThreads / 32];
    const int n = p.num_requests;
    int32_t* const starts = sums;
    int32_t* const offsets = sums + n + 1;
    pdl_wait_previous();
    pdl_release_next();
    const Split split(p.block_size);
    int32_t bits = 0;
    bool over = false;
    auto past_of = [&](int b) -> int64_t { return max(p.past[b], 0); };
    auto added_of = [&](int b) -> int64_t { return max(p.added[b], 0); };
    auto held_of = [&](int b) -> int64_t {
        return min(split.pages(past_of(b)), static_cast<int64_t>(p.table_width));
    };
    block_sums(n, starts, scratch, over, added_of);
    block_sums(n, offsets, scratch, over, [&](int b) -> int64_t {
        return min(split.pages(past_of(b) + added_of(b)), static_cast<int64_t>(p.table_width)) - held_of(b);
    });
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    const int64_t pages = offsets[n], total = starts[n];
    if (over) bits |= kErrSlot;
    for (int64_t b = first; b < n; b += step) {
        if (p.past[b] < 0 || p.added[b] < 0) bits |= kErrPos;
        p.starts[b] = starts[b];
    }
    if (first == 0) {
        p.starts[n] = starts[n];
        p.taken[0] = static_cast<int32_t>(min(pages, p.num_free));
        if (pages > p.num_free || total > p.num_tokens) bits |= kErrSlot;
    }
    for (int64_t j = first; j < min(pages, p.num_free); j += step) {
        const int b = find(offsets, n, static_cast<int32_t>(j));
        p.table[b * p.table_stride + held_of(b) + (j - offsets[b])] = p.free_pages[j];
    }
    for (int64_t row = first; row < p.num_tokens; row += step) {
        int64_t slot = -1, pos = 0;
        if (row < total) {
            const int b = find(starts, n, static_cast<int32_t>(row));
            pos = past_of(b) + (row - starts[b]);
            const int64_t page = split.page(static_cast<uint32_t>(pos)), held = held_of(b);
            int32_t id = -1;
            if (page < held) {
                id = p.table[b * p.table_stride + page];
            } else if (page < p.table_width) {
                const int64_t j = offsets[b] + (page - held);
                if (j < p.num_free) id = p.free_pages[j];
            }
            if (id >= 0) slot = static_cast<int64_t>(id) * p.block_size + (pos - page * p.block_size);
            else bits |= kErrSlot;
        }
        p.slots[row] = slot;
        p.positions[row] = pos;
    }
    if (bits != 0) report(p.err, bits);
}

// The slot of a position that request b holds, or -1 where the table has no page for it or the
// slot is no int32.
__device__ __forceinline__ int32_t slot_at(const SlotsParams& p, const Split& split, int64_t b, uint32_t pos,
                                           int32_t& bits) {
    const uint32_t page = split.page(pos);
    const int32_t id = page < static_cast<uint32_t>(p.table_width) ? p.table[b * p.table_stride + page] : -1;
    const int64_t slot = static_cast<int64_t>(id) * p.block_size + (pos - page * split.bs);
    if (id >= 0 && slot <= kIntMax) return static_cast<int32_t>(slot);
    bits |= kErrIndex;
    return -1;
}

__device__ __forceinline__ int64_t first_of(const SlotsParams& p, int64_t b) {
    return p.first == nullptr ? 0 : max(p.first[b], 0);
}
__device__ __forceinline__ int64_t count_of(const SlotsParams& p, int64_t b) {
    return max(static_cast<int64_t>(p.lengths[b]) - first_of(p, b), INT64_C(0));
}

// Rows of `width` entries, padded with -1: a block takes a run of one row.
constexpr int kRowEntries = 4;              // entries a thread
__global__ void __launch_bounds__(kPlanThreads) slots_kernel(const SlotsParams p, const int64_t parts) {
    pdl_wait_previous();
    pdl_release_next();
    const Split split(p.block_size);
    const int64_t b = blockIdx.x / parts, part = blockIdx.x - b * parts;
    const int64_t first = first_of(p, b), count = count_of(p, b);
    int32_t bits = 0;
    if (part == 0 && threadIdx.x == 0 &&
        (p.lengths[b] < 0 || (p.first != nullptr && p.first[b] < 0) || count > p.width))
        bits |= kErrIndex;
    int32_t* const out = p.indices + b * p.width;
#pragma unroll
    for (int i = 0; i < kRowEntries; ++i) {
        const int64_t at = (part * kRowEntries + i) * kPlanThreads + threadIdx.x;
        if (at >= p.width) break;
        out[at] = at < count ? slot_at(p, split, b, static_cast<uint32_t>(first + at), bits) : -1;
    }
    if (bits != 0) report(p.err, bits);
}

// One request after another, then -1.
__global__ void __launch_bounds__(kPlanThreads) packed_slots_kernel(const SlotsParams p) {
    extern __shared__ int32_t sums[];
    __shared__ int64_t scratch[kPlanThreads / 32];
    const int n = p.num_requests;
    pdl_wait_previous();
    pdl_release_next();
    const Split split(p.block_size);
    int32_t bits = 0;
    bool over = false;
    block_sums(n, sums, scratch, over, [&](int b) -> int64_t { return count_of(p, b); });
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    for (int64_t b = first; b <= n; b += step) {
        p.starts[b] = sums[b];
        if (b < n && (p.lengths[b] < 0 || (p.first != nullptr && p.first[b] < 0))) bits |= kErrIndex;
    }
    if (over || (first == 0 && sums[n] > p.width)) bits |= kErrIndex;
    for (int64_t row = first; row < p.width; row += step) {
        int32_t slot = -1;
        if (row < sums[n]) {
            const int b = find(sums, n, static_cast<int32_t>(row));
            slot = slot_at(p, split, b, static_cast<uint32_t>(first_of(p, b) + (row - sums[b])), bits);
        }
        p.indices[row] = slot;
    }
    if (bits != 0) report(p.err, bits);
}

// Shared memory for `arrays` arrays of num_requests + 1 sums: of two sizes only, so that the
// kernel's limit is set once and for good.
constexpr int kFewRequests = 4096;
size_t sums_bytes(int32_t num_requests, int arrays) {
    const int most = num_requests <= kFewRequests ? kFewRequests : kPlanMaxRequests;
    return arrays * (static_cast<size_t>(most) + 1) * sizeof(int32_t);
}

// Blocks of a launch over `rows` rows: a block for each kPlanThreads of them up to one wave,
// as every block sums the lengths first.
template <typename K>
cudaError_t plan_blocks(K kernel, size_t smem, int64_t rows, int64_t* blocks) {
    int64_t warps = 0;
    const cudaError_t e = resident_warps(reinterpret_cast<const void*>(kernel), kPlanThreads, smem, &warps);
    if (e != cudaSuccess) return e;
    const int64_t wave = warps / (kPlanThreads / 32), need = (rows + kPlanThreads - 1) / kPlanThreads;
    *blocks = need < 1 ? 1 : need < wave ? need : wave;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_allocate(const AllocateParams& p, cudaStream_t stream) {
    const size_t smem = sums_bytes(p.num_requests, 2);
    int64_t blocks = 0;
    const cudaError_t e = plan_blocks(allocate_kernel, smem, p.num_tokens, &blocks);
    if (e != cudaSuccess) return e;
    return launch_kernel(allocate_kernel, blocks, kPlanThreads, smem, stream, p.pdl, p);
}

cudaError_t launch_slots(const SlotsParams& p, cudaStream_t stream) {
    if (p.starts == nullptr) {
        constexpr int64_t kPer = kPlanThreads * kRowEntries;
        const int64_t parts = (p.width + kPer - 1) / kPer;
        return launch_kernel(slots_kernel, p.num_requests * parts, kPlanThreads, 0, stream, p.pdl, p, parts);
    }
    const size_t smem = sums_bytes(p.num_requests, 1);
    int64_t blocks = 0;
    const cudaError_t e = plan_blocks(packed_slots_kernel, smem, p.width, &blocks);
    if (e != cudaSuccess) return e;
    return launch_kernel(packed_slots_kernel, blocks, kPlanThreads, smem, stream, p.pdl, p);
}

}  // namespace gkr
