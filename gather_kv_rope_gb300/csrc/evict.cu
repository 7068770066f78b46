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
// unsigned key in the order of the values, and four passes, each counting the keys that share
// the bits found so far by their next 8 bits, fix those.  (Weights are few powers of two apart:
// eight copies of the counters, taken by the lane, keep most additions off each other's.)  Then each entry's fate is
// known -- kept if newer, or above that key, or equal to it and among the first `ties` such --
// and its place is a count of bits: entries are handled as words of 32 bits (live, competing,
// kept), one ballot each, and prefix sums run over the words.  Counts are whole numbers, so the
// result does not depend on the order of threads.
//
// A row is read once (8 bytes an entry; the kept and evicted slots a second time, from the
// caches): its keys stay in shared memory.  Long rows are split over a cluster of up to eight
// CTAs, which read each other's counts through distributed shared memory.  The work is a few
// microseconds of dependent steps, so latency bounds it, not memory.
#include "device.cuh"
#include "launch.h"
#include "tensor.cuh"

namespace gkr {

namespace {

constexpr int kBins = 256, kCopies = 8;
// Keys kept in shared memory up to this many entries a CTA; longer parts read the weights again
// for each pass.
constexpr int kCachedKeys = 36864;
constexpr int kMaxCluster = 8;

// A weight's key: unsigned order = order of the values; NaN 0 (below -inf), -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(__fadd_rn(w, 0.0f));
    return (b & 0x80000000u) != 0u ? ~b : (b | 0x80000000u);
}

// Exclusive prefix of v over the block's threads; *total = the sum.
template <int kThreads>
__device__ __forceinline__ int32_t block_prefix(int32_t v, int32_t* shared, int warp, int lane,
                                                int32_t* total) {
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();   // the last use of `shared` is over
    if (lane == 31) shared[warp] = x;
    __syncthreads();
    const int32_t w = lane < kThreads / 32 ? shared[lane] : 0;
    *total = __reduce_add_sync(kFull, w);
    return x - v + __reduce_add_sync(kFull, lane < warp ? w : 0);
}

// Exclusive prefix sums of the popcounts of bits[0 .. n) into out; returns their total.
template <int kThreads>
__device__ __forceinline__ int32_t scan_words(const uint32_t* bits, int32_t* out, int n,
                                              int32_t* shared, int warp, int lane) {
    const int per = (n + kThreads - 1) / kThreads;
    const int a = threadIdx.x * per, b = a + per < n ? a + per : n;
    int32_t sum = 0;
    for (int i = a; i < b; ++i) sum += __popc(bits[i]);
    int32_t total;
    int32_t x = block_prefix<kThreads>(sum, shared, warp, lane, &total);
    for (int i = a; i < b; ++i) {
        out[i] = x;
        x += __popc(bits[i]);
    }
    __syncthreads();
    return total;
}

// The lowest n set bits of x.
__device__ __forceinline__ uint32_t lowest_bits(uint32_t x, int32_t n) {
    if (n <= 0) return 0u;
    if (n >= __popc(x)) return x;
    return x & ((2u << __fns(x, 0, n)) - 1u);
}

__device__ __forceinline__ int32_t read_peer(const int32_t* p, uint32_t rank) {
    int32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_addr(p), rank)) : "memory");
    return v;
}

// Entries of words w0, w0 + step, ...: their slots (-1 past the part's end) and weights, all loads on
// their way before the first is used.
constexpr int kBatch = 8;
__device__ __forceinline__ void load_batch(const int32_t* idx, const float* wts, int w0, int step,
                                           int n, int32_t len, int lane, int32_t (&s)[kBatch],
                                           float (&x)[kBatch]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int32_t i = 32 * (w0 + step * u) + lane;
        const bool is = w0 + step * u < n && i < len;
        s[u] = is ? __ldg(idx + i) : -1;
        x[u] = is ? __ldg(wts + i) : 0.0f;
    }
}

struct alignas(16) EvictShared {
    int32_t scan[32];
    int32_t live, strict, tied;          // this CTA's counts, read by the others
    int32_t found[2];
    int32_t sum[4][kBins];               // counts, one array a pass: the others read it at their own time
    alignas(16) int32_t hist[kBins][kCopies];
};

// words: words of 32 entries of a CTA's part (the same for all CTAs of a row; the last may have
// less to do); cached: its keys lie in shared memory.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    evict_kernel(const EvictParams p, const int32_t words, const int32_t cluster, const bool cached) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    EvictShared& sh = *reinterpret_cast<EvictShared*>(dynamic);
    uint32_t* const live = reinterpret_cast<uint32_t*>(dynamic + sizeof(EvictShared));
    uint32_t* const some = live + words;                 // competing, then tied, then kept
    int32_t* const live_before = reinterpret_cast<int32_t*>(some + words);
    int32_t* const some_before = live_before + words;
    uint32_t* const keys = reinterpret_cast<uint32_t*>(some_before + words);
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = cluster > 1 ? cluster_rank() : 0u;
    const int64_t r = blockIdx.x / cluster;
    const int32_t e0 = static_cast<int32_t>(rank) * words * 32;
    const int32_t len = p.length - e0 < 0 ? 0 : p.length - e0 < words * 32 ? p.length - e0 : words * 32;
    const int32_t n = (len + 31) / 32;                   // words of this part
    pdl_wait_previous();
    pdl_release_next();
    const int32_t* const idx = p.indices + r * p.index_stride + e0;
    const float* const wts = p.weights + r * p.weight_stride + e0;
    auto sync = [&]() {                                  // and what was written is seen by the others
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    };
    // sum over the CTAs before this one, and over all, of a count
    auto exchange = [&](const int32_t* mine, int32_t* before) -> int32_t {
        if (cluster == 1) {
            *before = 0;
            return *mine;
        }
        const int32_t v = lane < cluster ? read_peer(mine, lane) : 0;
        *before = __reduce_add_sync(kFull, lane < static_cast<int>(rank) ? v : 0);
        return __reduce_add_sync(kFull, v);
    };

    for (int w0 = warp; w0 < n; w0 += kWarps * kBatch) {
        int32_t s[kBatch];
        float x[kBatch];
        load_batch(idx, wts, w0, kWarps, n, len, lane, s, x);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int w = w0 + kWarps * u;
            const uint32_t b = __ballot_sync(kFull, s[u] >= 0);
            if (w < n) {                                 // warp-uniform
                if (cached) keys[32 * w + lane] = s[u] >= 0 ? weight_key(x[u]) : 0u;
                if (lane == 0) live[w] = b;
            }
        }
    }
    __syncthreads();
    int32_t mine = scan_words<kThreads>(live, live_before, n, sh.scan, warp, lane);
    if (threadIdx.x == 0) sh.live = mine;
    sync();
    int32_t live0;                                       // live entries before this part
    const int32_t all = exchange(&sh.live, &live0);
    const int32_t fresh = p.recent < all ? p.recent : all;   // protected entries
    const int32_t old = all - fresh;                         // the first `old` live ones compete
    const int32_t room = p.keep - fresh < old ? p.keep - fresh : old;
    for (int w = threadIdx.x; w < n; w += kThreads)
        some[w] = lowest_bits(live[w], old - live0 - live_before[w]);
    __syncthreads();

    // the key of the last competing entry kept, and how many of its equals stay
    uint32_t key = 0, mask = 0;
    int32_t ties = room;
    if (room < old) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int i = threadIdx.x; i < kBins * kCopies; i += kThreads) sh.hist[0][i] = 0;
            __syncthreads();
            for (int w = warp; w < n; w += kWarps) {
                if ((some[w] >> lane & 1u) != 0u) {
                    const int32_t i = 32 * w + lane;
                    const uint32_t k = cached ? keys[i] : weight_key(__ldg(wts + i));
                    if ((k & mask) == key) atomicAdd(&sh.hist[k >> shift & 255u][lane & (kCopies - 1)], 1);
                }
            }
            __syncthreads();
            // bins from the top: thread t < 256 has bin 255 - t
            const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
            int32_t h = 0;
            if (bin >= 0) {
                const uint4 a = lds16(&sh.hist[bin][0]), b = lds16(&sh.hist[bin][4]);
                h = static_cast<int32_t>(a.x + a.y + a.z + a.w + b.x + b.y + b.z + b.w);
                sh.sum[pass][bin] = h;
            }
            if (cluster > 1) {
                sync();
                if (bin >= 0) {
                    int32_t v[kMaxCluster];
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c)   // all on their way before the first is used
                        v[c] = c < cluster ? read_peer(&sh.sum[pass][bin], c) : 0;
                    h = 0;
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c) h += v[c];
                }
            }
            int32_t total;
            const int32_t above = block_prefix<kThreads>(h, sh.scan, warp, lane, &total);
            // the first bin, from the top, that brings the count to `ties` (to more than 0 where
            // that is 0: nothing is kept, and the top bin serves)
            const int32_t want = ties > 0 ? ties : 1;
            if (above < want && above + h >= want) {
                sh.found[0] = bin;
                sh.found[1] = ties - above;
            }
            __syncthreads();
            key |= static_cast<uint32_t>(sh.found[0]) << shift;
            mask |= 255u << shift;
            ties = sh.found[1];
            __syncthreads();
        }
    }

    // competing entries above the key, and those equal to it
    int32_t strict = 0, tied = 0;
    if (room < old) {
        for (int w = warp; w < n; w += kWarps) {
            const uint32_t c = some[w];
            const int32_t i = 32 * w + lane;
            const bool is = (c >> lane & 1u) != 0u;
            const uint32_t k = !is ? 0u : cached ? keys[i] : weight_key(__ldg(wts + i));
            const uint32_t above = __ballot_sync(kFull, is && k > key);
            const uint32_t equal = __ballot_sync(kFull, is && k == key);
            __syncwarp();
            if (lane == 0) {
                some[w] = equal;
                some_before[w] = static_cast<int32_t>(above | (live[w] & ~c));   // bits kept in any case
            }
            strict += __popc(above | (live[w] & ~c));
            tied += __popc(equal);
        }
    }
    // totals of this CTA (each word was counted by all lanes of one warp)
    __syncthreads();
    if (threadIdx.x == 0) {
        sh.strict = 0;
        sh.tied = 0;
    }
    __syncthreads();
    if (lane == 0 && room < old) {
        atomicAdd(&sh.strict, strict);
        atomicAdd(&sh.tied, tied);
    }
    __syncthreads();
    int32_t kept0 = 0;                                   // kept entries before this part
    if (room < old) {
        sync();
        // before: the other CTAs' strictly kept entries, and of their ties what still had room
        int32_t tied0;
        exchange(&sh.tied, &tied0);
        if (cluster > 1) {
            int32_t strict0;
            exchange(&sh.strict, &strict0);
            kept0 = strict0 + (tied0 < ties ? tied0 : ties);
        }
        // this part's ties in order; then the kept words
        int32_t run = tied0;
        for (int w0 = 0; w0 < n; w0 += kThreads) {
            const int w = w0 + threadIdx.x;
            const uint32_t equal = w < n ? some[w] : 0u;
            int32_t total;
            const int32_t x = run + block_prefix<kThreads>(__popc(equal), sh.scan, warp, lane, &total);
            run += total;
            if (w < n) some[w] = static_cast<uint32_t>(some_before[w]) | lowest_bits(equal, ties - x);
        }
        __syncthreads();
    } else {                                             // every live entry stays
        for (int w = threadIdx.x; w < n; w += kThreads) some[w] = live[w];
        kept0 = live0;
        __syncthreads();
    }
    scan_words<kThreads>(some, some_before, n, sh.scan, warp, lane);

    int32_t* const kept = p.kept + r * p.keep;
    float* const kept_w = p.kept_weights + r * p.keep;
    int64_t* const gone = p.evicted + r * (p.length - p.keep);
    for (int w0 = warp; w0 < n; w0 += kWarps * kBatch) {
        int32_t s[kBatch];
        float x[kBatch];
        load_batch(idx, wts, w0, kWarps, n, len, lane, s, x);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int w = w0 + kWarps * u;
            if (w < n && s[u] >= 0) {
                const uint32_t l = live[w], k = some[w], below = (1u << lane) - 1u;
                const int32_t a = kept0 + some_before[w] + __popc(k & below);
                if ((k >> lane & 1u) != 0u) {
                    kept[a] = s[u];
                    kept_w[a] = x[u];
                } else {
                    gone[live0 + live_before[w] + __popc(l & below) - a] = s[u];
                }
            }
        }
    }
    // what is left of the row's outputs, spread over its CTAs
    const int32_t kept_all = fresh + room;
    for (int32_t i = kept_all + rank * kThreads + threadIdx.x; i < p.keep; i += cluster * kThreads) {
        kept[i] = -1;
        kept_w[i] = 0.0f;
    }
    for (int32_t i = all - kept_all + rank * kThreads + threadIdx.x; i < p.length - p.keep;
         i += cluster * kThreads)
        gone[i] = -1;
    if (cluster > 1) cluster_sync();                     // no CTA leaves while another reads its counts
}

template <int kThreads>
cudaError_t launch(const EvictParams& p, int32_t cluster, cudaStream_t stream) {
    const int32_t words = (p.length + 32 * cluster - 1) / (32 * cluster);
    const bool cached = words * 32 <= kCachedKeys;
    const size_t smem = sizeof(EvictShared) + static_cast<size_t>(words) * (cached ? 16 + 128 : 16);
    // raises the kernel's limit once per device
    int64_t warps = 0;
    const cudaError_t e = resident_warps(reinterpret_cast<const void*>(evict_kernel<kThreads>), kThreads,
                                         sizeof(EvictShared) + kCachedKeys / 32 * 144, &warps);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = p.pdl != 0 ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel<kThreads>, p, words, cluster, cached);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    // CTAs a row: one for each 8192 entries, at most eight; few threads wait less for each other
    // where the entries are few
    int32_t cluster = 1;
    while (cluster < kMaxCluster && p.length > 8192 * cluster) cluster *= 2;
    return p.length <= 4096 ? launch<256>(p, 1, stream) : launch<1024>(p, cluster, stream);
}

}  // namespace gkr
