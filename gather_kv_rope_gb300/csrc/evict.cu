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
// unsigned key in the order of the values, and up to four passes, each counting the keys that
// share the bits found so far by their next 8 bits, fix those, until all keys that share them
// stay.  (Weights are few powers of two apart: eight copies of the counters, taken by the lane,
// keep most additions off each other's.)  Then each entry's fate is known -- kept if newer, or
// above that key, or equal to it and among the first `ties` such -- and its place is a count of
// bits: entries are handled as words of 32 bits (live, competing, kept), and prefix sums run over
// the words.  Counts are whole numbers, so the result does not depend on the order of threads.
//
// A row is read once (8 bytes an entry; the kept weights a second time): its keys and slots stay
// in shared memory.  Long rows are split over a cluster of up to eight CTAs, which read each
// other's counts through distributed shared memory.  The work is a few dependent steps on little
// data, so their latency and the instructions of a few CTAs bound it, not memory: with one entry a
// lane and instruction a step over 16384 entries of a CTA took 3600 cycles (25 instructions for
// 32 entries), so a lane takes four at a time where it can.  Measured in a graph (weights of a
// log-normal distribution, a tenth of them zeros; in brackets uniform ones to the fourth power):
// keeping 4096 of 4 x 131071 entries 22 us (24), 2048 of 128 x 2049 9.1 us (7.0), 65536 of
// 16 x 1000000 312 us (317).
#include "device.cuh"
#include "launch.h"
#include "tensor.cuh"

namespace gkr {

namespace {

constexpr int kBins = 256, kCopies = 8;
// Keys, and slots, kept in shared memory up to this many entries a CTA; longer parts read the
// weights again for each pass, and the slots when they leave.
constexpr int kCachedKeys = 36864, kCachedSlots = 20480;
constexpr size_t kMostWords = kCachedSlots / 32 * (16 + 256);   // bytes
static_assert(kCachedKeys / 32 * (16 + 128) <= kMostWords, "fits where keys and slots do");
constexpr int kMaxCluster = 8, kFewEntries = 2560;

// A weight's key: unsigned order = order of the values; NaN 1 (below -inf, 2^23 - 1), -0 as 0.
// What does not compete has key 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 1u;
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

// A word of 32 entries: which are live; which compete, then tie, then are kept; and how many
// live, and kept, ones come before it.
struct alignas(16) Word {
    uint32_t live, some;
    int32_t live_before, some_before;
};

// Exclusive prefix sums of the popcounts of a field of word[0 .. n) into another; returns their
// total.
template <int kThreads>
__device__ __forceinline__ int32_t scan_words(Word* word, uint32_t Word::* bits, int32_t Word::* out, int n,
                                              int32_t* shared, int warp, int lane) {
    const int per = (n + kThreads - 1) / kThreads;
    const int a = threadIdx.x * per, b = a + per < n ? a + per : n;
    int32_t sum = 0;
    for (int i = a; i < b; ++i) sum += __popc(word[i].*bits);
    int32_t total;
    int32_t x = block_prefix<kThreads>(sum, shared, warp, lane, &total);
    for (int i = a; i < b; ++i) {
        word[i].*out = x;
        x += __popc(word[i].*bits);
    }
    __syncthreads();
    return total;
}

// Four bits of each lane as the words of eight lanes each: all eight get theirs.
__device__ __forceinline__ uint32_t word_of_nibbles(uint32_t nibble, int lane) {
    uint32_t x = nibble << (4 * (lane & 7));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) x |= __shfl_xor_sync(kFull, x, d);
    return x;
}

// Entries i .. i + 3 of a row, `none` past its end.
template <typename V4, typename T>
__device__ __forceinline__ V4 load4(const T* row, int32_t i, int32_t len, bool aligned, T none) {
    V4 v;
    if (aligned && i + 4 <= len) {
        v = __ldg(reinterpret_cast<const V4*>(row + i));
    } else {
        v.x = i < len ? __ldg(row + i) : none;
        v.y = i + 1 < len ? __ldg(row + i + 1) : none;
        v.z = i + 2 < len ? __ldg(row + i + 2) : none;
        v.w = i + 3 < len ? __ldg(row + i + 3) : none;
    }
    return v;
}

// The lowest n set bits of x.
__device__ __forceinline__ uint32_t lowest_bits(uint32_t x, int32_t n) {
    if (n <= 0) return 0u;
    if (n >= __popc(x)) return x;
    int p = 0;   // the highest place with at most n bits below it
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1)
        if (__popc(x & ((1u << (p + step)) - 1u)) <= n) p += step;
    return x & ((1u << p) - 1u);
}

__device__ __forceinline__ int32_t read_peer(const int32_t* p, uint32_t rank) {
    int32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_addr(p), rank)) : "memory");
    return v;
}

constexpr int kBatch = 4;   // groups of four words (at the end: words) of a warp in flight

struct alignas(16) EvictShared {
    int32_t scan[32];
    int32_t live, strict, tied;          // this CTA's counts, read by the others
    int32_t found[3];
    int32_t sum[4][kBins];               // counts, one array a pass: the others read it at their own time
    alignas(16) int32_t hist[kBins][kCopies];
};

// words: words of 32 entries of a CTA's part (the same for all CTAs of a row; the last may have
// less to do); its keys, and its slots, lie in shared memory where they are `cached`.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    evict_kernel(const EvictParams p, const int32_t words, const int32_t cluster,
                 const bool keys_cached, const bool slots_cached) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    EvictShared& sh = *reinterpret_cast<EvictShared*>(dynamic);
    Word* const word = reinterpret_cast<Word*>(dynamic + sizeof(EvictShared));
    uint32_t* const keys = reinterpret_cast<uint32_t*>(word + words);
    int32_t* const slots = reinterpret_cast<int32_t*>(keys + 32 * words);
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = cluster > 1 ? cluster_rank() : 0u;
    const int64_t r = blockIdx.x / cluster;
    const int32_t e0 = static_cast<int32_t>(rank) * words * 32;
    const int32_t len = p.length - e0 < 0 ? 0 : p.length - e0 < words * 32 ? p.length - e0 : words * 32;
    const int32_t n = (len + 127) / 128 * 4;             // words of this part
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

    const bool aligned = ((reinterpret_cast<uintptr_t>(idx) | reinterpret_cast<uintptr_t>(wts)) & 15) == 0;
    // The keys of words w .. w + 3, four a lane.
    auto load_keys = [&](int w) -> uint4 {
        const int32_t i = 32 * w + 4 * lane;
        if (keys_cached) return lds16(keys + i);
        const uint32_t c = word[w + (lane >> 3)].some >> (4 * (lane & 7));
        const float4 x = load4<float4, float>(wts, i, len, aligned, 0.0f);
        return make_uint4((c & 1u) != 0u ? weight_key(x.x) : 0u, (c & 2u) != 0u ? weight_key(x.y) : 0u,
                          (c & 4u) != 0u ? weight_key(x.z) : 0u, (c & 8u) != 0u ? weight_key(x.w) : 0u);
    };

    for (int w0 = 4 * warp; w0 < n; w0 += 4 * kWarps * kBatch) {
        int4 s[kBatch];
        float4 x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t i = 32 * (w0 + 4 * kWarps * u) + 4 * lane;
            s[u] = load4<int4, int32_t>(idx, i, len, aligned, -1);
            if (keys_cached) x[u] = load4<float4, float>(wts, i, len, aligned, 0.0f);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int w = w0 + 4 * kWarps * u;
            if (w < n) {                                 // warp-uniform
                const bool a = s[u].x >= 0, b = s[u].y >= 0, c = s[u].z >= 0, d = s[u].w >= 0;
                const int32_t i = 32 * w + 4 * lane;
                if (keys_cached)
                    *reinterpret_cast<uint4*>(keys + i) =
                        make_uint4(a ? weight_key(x[u].x) : 0u, b ? weight_key(x[u].y) : 0u,
                                   c ? weight_key(x[u].z) : 0u, d ? weight_key(x[u].w) : 0u);
                if (slots_cached) *reinterpret_cast<int4*>(slots + i) = s[u];
                const uint32_t bits = word_of_nibbles((a ? 1u : 0u) | (b ? 2u : 0u) | (c ? 4u : 0u) | (d ? 8u : 0u), lane);
                if ((lane & 7) == 0) word[w + (lane >> 3)].live = bits;
            }
        }
    }
    __syncthreads();
    int32_t mine = scan_words<kThreads>(word, &Word::live, &Word::live_before, n, sh.scan, warp, lane);
    if (threadIdx.x == 0) sh.live = mine;
    sync();
    int32_t live0;                                       // live entries before this part
    const int32_t all = exchange(&sh.live, &live0);
    const int32_t fresh = p.recent < all ? p.recent : all;   // protected entries
    const int32_t old = all - fresh;                         // the first `old` live ones compete
    const int32_t room = p.keep - fresh < old ? p.keep - fresh : old;
    for (int w = threadIdx.x; w < n; w += kThreads) {
        const uint32_t l = word[w].live, c = lowest_bits(l, old - live0 - word[w].live_before);
        word[w].some = c;
    }
    __syncthreads();
    if (keys_cached && live0 + mine > old) {             // protected entries do not compete
        for (int w = warp; w < n; w += kWarps)
            if (((word[w].live & ~word[w].some) >> lane & 1u) != 0u) keys[32 * w + lane] = 0u;
    }

    // the key of the last competing entry kept, and how many of its equals stay
    uint32_t key = 0, mask = 0;
    int32_t ties = room;
    if (room < old) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int i = threadIdx.x; i < kBins * kCopies; i += kThreads) sh.hist[0][i] = 0;
            __syncthreads();
            auto count = [&](uint32_t k) {
                if ((k & mask) == key) atomicAdd(&sh.hist[k >> shift & 255u][lane & (kCopies - 1)], 1);
            };
#pragma unroll 2
            for (int w = 4 * warp; w < n; w += 4 * kWarps) {
                const uint4 k = load_keys(w);
                count(k.x);
                count(k.y);
                count(k.z);
                count(k.w);
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
                sh.found[2] = h;
            }
            __syncthreads();
            key |= static_cast<uint32_t>(sh.found[0]) << shift;
            mask |= 255u << shift;
            ties = sh.found[1];
            const bool whole = sh.found[2] == ties;      // every key that begins like this one stays:
            __syncthreads();                             // its other bits do not matter
            if (whole) break;
        }
    }

    // competing entries above the key, and those equal to it, in the bits that were fixed
    int32_t strict = 0, tied = 0;
    if (room < old) {
#pragma unroll 2
        for (int w0 = 4 * warp; w0 < n; w0 += 4 * kWarps) {
            const uint4 k4 = load_keys(w0);
            const uint32_t k[4] = {k4.x & mask, k4.y & mask, k4.z & mask, k4.w & mask};
            uint32_t above = 0u, equal = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                above |= k[i] > key ? 1u << i : 0u;
                equal |= k[i] == key ? 1u << i : 0u;
            }
            above = word_of_nibbles(above, lane);
            equal = word_of_nibbles(equal, lane);
            if ((lane & 7) == 0) {
                Word& w = word[w0 + (lane >> 3)];
                const uint32_t c = w.some, stay = (above & c) | (w.live & ~c);   // kept in any case
                equal &= c;
                w.some = equal;
                w.some_before = static_cast<int32_t>(stay);
                strict += __popc(stay);
                tied += __popc(equal);
            }
        }
    }
    // totals of this CTA
    strict = __reduce_add_sync(kFull, strict);
    tied = __reduce_add_sync(kFull, tied);
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
            const uint32_t equal = w < n ? word[w].some : 0u;
            int32_t total;
            const int32_t x = run + block_prefix<kThreads>(__popc(equal), sh.scan, warp, lane, &total);
            run += total;
            if (w < n) word[w].some = static_cast<uint32_t>(word[w].some_before) | lowest_bits(equal, ties - x);
        }
        __syncthreads();
    } else {                                             // every live entry stays
        for (int w = threadIdx.x; w < n; w += kThreads) word[w].some = word[w].live;
        kept0 = live0;
        __syncthreads();
    }
    scan_words<kThreads>(word, &Word::some, &Word::some_before, n, sh.scan, warp, lane);

    int32_t* const kept = p.kept + r * p.keep;
    float* const kept_w = p.kept_weights + r * p.keep;
    int64_t* const gone = p.evicted + r * (p.length - p.keep);
    const uint32_t below = (1u << lane) - 1u;
    for (int w0 = warp; w0 < n; w0 += kWarps * kBatch) {
        uint4 x[kBatch];
        int32_t s[kBatch];
        float weight[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int w = w0 + kWarps * u;
            const int32_t i = 32 * w + lane;
            x[u] = w < n ? lds16(word + w) : make_uint4(0u, 0u, 0u, 0u);
            const bool is = (x[u].x >> lane & 1u) != 0u;
            s[u] = !is ? -1 : slots_cached ? slots[i] : __ldg(idx + i);
            weight[u] = (x[u].y >> lane & 1u) != 0u ? __ldg(wts + i) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t before = kept0 + static_cast<int32_t>(x[u].w) + __popc(x[u].y & below);
            if ((x[u].y >> lane & 1u) != 0u) {
                kept[before] = s[u];
                kept_w[before] = weight[u];
            } else if (s[u] >= 0) {
                gone[live0 + static_cast<int32_t>(x[u].z) + __popc(x[u].x & below) - before] = s[u];
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
    const int32_t words = (p.length + 128 * cluster - 1) / (128 * cluster) * 4;
    const bool keys_cached = words * 32 <= kCachedKeys, slots_cached = words * 32 <= kCachedSlots;
    const size_t smem = sizeof(EvictShared) +
                        static_cast<size_t>(words) * (16 + (keys_cached ? 128 : 0) + (slots_cached ? 128 : 0));
    // raises the kernel's limit once per device
    int64_t warps = 0;
    const cudaError_t e = resident_warps(reinterpret_cast<const void*>(evict_kernel<kThreads>), kThreads,
                                         sizeof(EvictShared) + kMostWords, &warps);
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
    return cudaLaunchKernelEx(&cfg, evict_kernel<kThreads>, p, words, cluster, keys_cached,
                              slots_cached);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    // CTAs a row: as many as it takes to keep a part's keys in shared memory, then more, down to 4096
    // entries each, while all rows' CTAs run at once (128 of the 152 SMs: whole clusters have
    // to fit).  Measured, us in a graph, half of the entries kept: 4 rows x 16384 entries 16.2
    // with one CTA a row, 14.5 with two, 12.3 with four, 12.5 with eight; 4 x 32768 26.9, 19.4, 14.9 and
    // 13.9; 64 x 16384 17.5 with one, 16.1 with two, 26.7 with four; 64 x 32768 28.9, 21.6 and 31.9;
    // 64 x 65536 33.4 with two, 42.3 with four, 84.1 with eight.
    int32_t cluster = 1;
    while (cluster < kMaxCluster &&
           (p.length > kCachedKeys * cluster || (p.length > 4096 * cluster && p.rows * cluster * 2 <= 128)))
        cluster *= 2;
    // few threads wait less for each other where the entries are few: 128 rows x 1024 entries, half
    // kept, 5.8 us with 256 threads and 7.8 with 1024, x 2049 8.7 and 9.0, x 4096 10.5 and 9.7
    return p.length <= kFewEntries ? launch<256>(p, 1, stream) : launch<1024>(p, cluster, stream);
}

}  // namespace gkr
