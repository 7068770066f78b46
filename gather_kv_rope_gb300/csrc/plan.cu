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
// The outputs are a few bytes a token, so latencies bound all but the largest calls, and one launch
// does everything: every block sums the lengths of all requests for itself (a few KB from L2) and
// then finds the request of each of its rows by bisection in shared memory.  Measured in a graph:
// decoding 64 requests 3.5 to 3.7 us, 524288 tokens of 512 requests 7.5 to 7.8 (their bytes take 1.2), 64 lists
// of 8191 slots 2.5 to 3.0, 8 packed ones of up to 131072 4.9 to 5.0; a call from Python takes 10 to 26, the
// host's time.
// New pages are read from the free list, not from the table that other blocks are writing.  No atomics but
// for the error bits: the same call gives the same bytes.
#include "device.cuh"
#include "launch.h"

namespace gkr {

namespace {

constexpr int32_t kErrSlot = 1, kErrPos = 2, kErrIndex = 4;
constexpr int kPlanThreads = 512;
constexpr int64_t kIntMax = INT64_C(0x7FFFFFFF);

// Two sums at a time.
struct Pair {
    int64_t a, b;
    __device__ Pair operator+(const Pair& o) const { return {a + o.a, b + o.b}; }
    __device__ Pair operator-(const Pair& o) const { return {a - o.a, b - o.b}; }
};
__device__ __forceinline__ Pair warp_inclusive(Pair v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Pair o = {__shfl_up_sync(kFull, v.a, d), __shfl_up_sync(kFull, v.b, d)};
        if (lane >= d) v = v + o;
    }
    return v;
}

// Exclusive sums of f(0) .. f(n - 1), whose parts are each at most kIntMax, into a[0 .. n] and b[0 .. n]
// (clamped to kIntMax: `over` tells).  Each thread sums a run of consecutive elements.
template <typename F>
__device__ void block_sums(int n, int32_t* a, int32_t* b, Pair* scratch, bool& over, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int run = (n + kPlanThreads - 1) / kPlanThreads;
    const int first = min(n, static_cast<int>(threadIdx.x) * run), last = min(n, first + run);
    Pair sum = {0, 0}, one = {0, 0};        // one: the only element, if there is one
    for (int i = first; i < last; ++i) {
        one = f(i);
        sum = sum + one;
    }
    const Pair upto = warp_inclusive(sum, lane);
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    // every warp sums the warps before it
    Pair at = lane < warp ? scratch[lane] : Pair{0, 0};
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        at = at + Pair{__shfl_xor_sync(kFull, at.a, d), __shfl_xor_sync(kFull, at.b, d)};
    at = at + upto - sum;
    for (int i = first; i < last; ++i) {
        a[i] = static_cast<int32_t>(min(at.a, kIntMax));
        b[i] = static_cast<int32_t>(min(at.b, kIntMax));
        at = at + (run == 1 ? one : f(i));
    }
    if (last == n && (first < n || threadIdx.x == 0)) {   // the thread of the last element
        a[n] = static_cast<int32_t>(min(at.a, kIntMax));
        b[n] = static_cast<int32_t>(min(at.b, kIntMax));
        over = at.a > kIntMax || at.b > kIntMax;
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

// A thread takes kRun consecutive rows: one bisection, and one page for as long as they lie in it.  One
// row where there are threads for all: decoding 64 requests takes 3.5 us with one, 5.9 with four, 512
// requests 4.1 and 7.0; 512 requests of 1024 tokens 7.9 and 7.4, of 8192 34 and 29, 16384 of 512 186 and 124.
constexpr int64_t kLongRun = 4;
template <int kRun>
__global__ void __launch_bounds__(kPlanThreads) allocate_kernel(const AllocateParams p) {
    extern __shared__ int32_t sums[];       // starts[n + 1], offsets[n + 1]
    __shared__ Pair scratch[kPlanThreads / 32];
    const int n = p.num_requests;
    int32_t* const starts = sums;
    int32_t* const offsets = sums + n + 1;
    pdl_wait_previous();
    pdl_release_next();
    const Split split(p.block_size);
    int32_t bits = 0;
    bool over = false;
    auto past_of = [&](int b) -> int64_t { return max(p.past[b], 0); };
    auto held_of = [&](int b) -> int64_t {
        return min(split.pages(past_of(b)), static_cast<int64_t>(p.table_width));
    };
    block_sums(n, starts, offsets, scratch, over, [&](int b) -> Pair {
        const int64_t past = past_of(b), added = max(p.added[b], 0), width = p.table_width;
        return {added, min(split.pages(past + added), width) - min(split.pages(past), width)};
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
    const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
    for (int64_t row0 = first * kRun; row0 < p.num_tokens; row0 += step * kRun) {
        int64_t slot[kRun], pos[kRun];
        int b = -1;
        int64_t page = -1, id = -1;         // of the row before
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int64_t row = row0 + i;
            slot[i] = -1;
            pos[i] = 0;
            if (row >= total) continue;
            if (b < 0 || row >= starts[b + 1]) {
                b = find(starts, n, static_cast<int32_t>(row));
                page = -1;
            }
            pos[i] = past_of(b) + (row - starts[b]);
            const int64_t mine = split.page(static_cast<uint32_t>(pos[i]));
            if (mine != page) {
                page = mine;
                const int64_t held = held_of(b);
                id = -1;
                if (page < held) {
                    id = p.table[b * p.table_stride + page];
                } else if (page < p.table_width) {
                    const int64_t j = offsets[b] + (page - held);
                    if (j < p.num_free) id = p.free_pages[j];
                }
            }
            if (id >= 0) slot[i] = id * p.block_size + (pos[i] - page * p.block_size);
            else if (row < p.num_tokens) bits |= kErrSlot;
        }
        if (kRun > 1 && wide && row0 + kRun <= p.num_tokens) {
#pragma unroll
            for (int i = 0; i + 1 < kRun; i += 2) {
                *reinterpret_cast<longlong2*>(p.slots + row0 + i) = make_longlong2(slot[i], slot[i + 1]);
                *reinterpret_cast<longlong2*>(p.positions + row0 + i) = make_longlong2(pos[i], pos[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                if (row0 + i >= p.num_tokens) break;
                p.slots[row0 + i] = slot[i];
                p.positions[row0 + i] = pos[i];
            }
        }
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

// One request after another, then -1; kRun consecutive entries a thread, as above.
template <int kRun>
__global__ void __launch_bounds__(kPlanThreads) packed_slots_kernel(const SlotsParams p) {
    extern __shared__ int32_t sums[];       // starts[n + 1], and as much for the other sum
    __shared__ Pair scratch[kPlanThreads / 32];
    const int n = p.num_requests;
    int32_t* const starts = sums;
    pdl_wait_previous();
    pdl_release_next();
    const Split split(p.block_size);
    int32_t bits = 0;
    bool over = false;
    block_sums(n, starts, sums + n + 1, scratch, over, [&](int b) -> Pair { return {count_of(p, b), 0}; });
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    const int64_t total = starts[n];
    for (int64_t b = first; b <= n; b += step) {
        p.starts[b] = starts[b];
        if (b < n && (p.lengths[b] < 0 || (p.first != nullptr && p.first[b] < 0))) bits |= kErrIndex;
    }
    if (over || (first == 0 && total > p.width)) bits |= kErrIndex;
    const bool wide = (reinterpret_cast<uintptr_t>(p.indices) & 15) == 0;
    for (int64_t row0 = first * kRun; row0 < p.width; row0 += step * kRun) {
        int32_t slot[kRun];
        int b = -1;
        int64_t from = 0;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int64_t row = row0 + i;
            slot[i] = -1;
            if (row >= total || row >= p.width) continue;
            if (b < 0 || row >= starts[b + 1]) {
                b = find(starts, n, static_cast<int32_t>(row));
                from = first_of(p, b) - starts[b];
            }
            slot[i] = slot_at(p, split, b, static_cast<uint32_t>(from + row), bits);
        }
        if (kRun == 4 && wide && row0 + kRun <= p.width) {
            *reinterpret_cast<int4*>(p.indices + row0) = make_int4(slot[0], slot[1 % kRun], slot[2 % kRun], slot[3 % kRun]);
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (row0 + i < p.width) p.indices[row0 + i] = slot[i];
        }
    }
    if (bits != 0) report(p.err, bits);
}

// Shared memory for two arrays of num_requests + 1 sums: of two sizes only, so that the
// kernel's limit is set once and for good.
constexpr int kFewRequests = 4096;
size_t sums_bytes(int32_t num_requests) {
    const int most = num_requests <= kFewRequests ? kFewRequests : kPlanMaxRequests;
    return 2 * (static_cast<size_t>(most) + 1) * sizeof(int32_t);
}

// One row a thread where one wave has threads for all, else runs, in one wave at most, as every block sums
// the lengths first.
template <typename P>
cudaError_t launch_rows(void (*one)(P), void (*runs)(P), const P& p, int64_t rows, cudaStream_t stream) {
    const size_t smem = sums_bytes(p.num_requests);
    int64_t warps = 0;
    cudaError_t e = resident_warps(reinterpret_cast<const void*>(one), kPlanThreads, smem, &warps);
    if (e != cudaSuccess) return e;
    if (rows <= warps * 32) {
        const int64_t blocks = (rows + kPlanThreads - 1) / kPlanThreads;
        return launch_kernel(one, blocks < 1 ? 1 : blocks, kPlanThreads, smem, stream, p.pdl, p);
    }
    e = resident_warps(reinterpret_cast<const void*>(runs), kPlanThreads, smem, &warps);
    if (e != cudaSuccess) return e;
    const int64_t wave = warps / (kPlanThreads / 32), per = kPlanThreads * kLongRun, need = (rows + per - 1) / per;
    return launch_kernel(runs, need < wave ? need : wave, kPlanThreads, smem, stream, p.pdl, p);
}

}  // namespace

cudaError_t launch_allocate(const AllocateParams& p, cudaStream_t stream) {
    return launch_rows(allocate_kernel<1>, allocate_kernel<kLongRun>, p, p.num_tokens, stream);
}

cudaError_t launch_slots(const SlotsParams& p, cudaStream_t stream) {
    if (p.starts == nullptr) {
        constexpr int64_t kPer = kPlanThreads * kRowEntries;
        const int64_t parts = p.width > 0 ? (p.width + kPer - 1) / kPer : 1;   // 1: only errors, no entries
        return launch_kernel(slots_kernel, p.num_requests * parts, kPlanThreads, 0, stream, p.pdl, p, parts);
    }
    return launch_rows(packed_slots_kernel<1>, packed_slots_kernel<kLongRun>, p, p.width, stream);
}

}  // namespace gkr
