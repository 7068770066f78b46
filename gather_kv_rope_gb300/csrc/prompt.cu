// Attention of packed requests over packed bf16 latent rows, and decode attention of a batch
// behind a shared prefix of MXFP4 records.
//
// Operation (the latent row is key and value of every head, as in the sparse attention): a
// query head q that sees the rows K[0 .. see - 1] of its request gets
//   s[k] = sm_scale * q . K[k],  m = max s,  l = sum exp(s - m),
//   out = sum exp(s[k] - m) K[k] / l,  lse = m + log l;   see = 0: zeros and -inf.
// Causal: of a request's n queries and m rows, query i sees m - n + i + 1.
//
// A request's query heads are rows of one matrix, query after query, and a tile is 128 of them,
// whatever the number of heads: 128 heads of one query or 16 of eight.  A pair of CTAs
// (cta_group::2, M = 128) multiplies a tile by chunks of 128 rows of K, both products, 2 x 128 x
// 128 x 512 multiply-adds: 2048 cycles of the two SMs' tensor cores.  They are the floor of
// every larger call, so everything else runs beside them:
//   * The accumulator, 128 x 512 fp32, takes half of the two SMs' tensor memory, a chunk's logits
//     an eighth (64 columns), three quarters of the query tile the rest (192 columns).
//   * Rows come by TMA into a ring of three stages of 64 KB: a CTA's own 64 rows of the chunk for
//     q . K; once that is done, the half of the dims that the other CTA multiplies is replaced
//     by the other 64 rows' half of this CTA's dims for p . K (a product of the pair takes half
//     of its columns from each CTA, at the same address in both).
//   * The next query tile passes through the ring like a chunk; the tensor cores copy it on to
//     tensor memory (tcgen05.cp).  Its stage then takes the results of the tile before, which leave
//     by TMA stores of eight warps of their own.  So neither is on the softmax's way, and little of
//     it on that of the warps' loads, stores and tensor-memory accesses: one pipe of 128 bytes a
//     cycle, which a tile's query and results took for 9000 cycles.
//   * q . K of the next chunk is issued before p . K of this one, so that the softmax of a chunk
//     has the time of two products.  The probabilities have one buffer, and so have the logits.
//   * The thread that issues the products waits for one barrier before each, at which the softmax
//     and a warp of each CTA that relays what has landed arrive: three barriers took 400
//     cycles a chunk.  Its loops are unrolled: rolled up they cost a quarter of the rate.
//   * Work: units for each tile (its loads and its epilogue, as long as two chunks) and for each of
//     its chunks, all tiles in a row, cut evenly over the pairs.  One warp of each CTA finds the cut
//     from the requests' lengths by itself (closed sums, no plan to launch).  The pieces of a tile
//     that is cut go to the workspace (fp32 rows and their log-sum-exp) and a second kernel joins
//     them.  Where there are few tiles and none much longer than an even share, each pair has
//     a whole one; that is looked at for up to 32 requests, one a lane, while more are always cut (one
//     query of 128 heads and 300 rows a request: 32 requests 14.7 us, 33 20.4, 64 25.2; 1500
//     rows: 28.1, 30.3, 47.1).  A share of more than 131072 rows is taken in runs (kRunChunks).
// The tensor cores take the probabilities as bf16 (A and B of a product have one type, and the rows are
// bf16).  The reference lags the maximum, so the largest one is no power of two, and where one row of K has
// most of the weight its rounding, up to 2^-9, is the result's as well.  So results are divided by the
// sum of the probabilities as they were rounded, in which such a rounding cancels, and only the
// log-sum-exp comes from the sum of what was not: the results of 128 queries of 128 heads behind 16384
// records are then 0.0017 off (root mean square, relative; rounding them to bf16 alone takes 0.0016), before it
// was 0.0022.  It costs 1.3 % where the power cap is near (8192 x 64 heads 2.25 -> 2.28 ms), else
// nothing (4096 x 64 0.627 and 0.625), as the second sum is taken once the products may begin.
// What a row does not see: columns past its last row are -inf before the softmax.  Their
// probabilities are 0, but 0 times an infinity or NaN is NaN, so in a chunk with such
// columns, values that are not finite are cleared before p . K.  A row that does see them has NaN from
// its logit, unless that is -inf: then its result is finite, where in a chunk that every row of the tile
// sees in full, and that nothing is cleared in, it is NaN.
//
// Measured (in a graph): 8192 tokens of 64 heads 2.27 to 2.36 ms, 1940 to 1865 TFLOP/s, 99 to 95 % of the
// measured burst rate (at the power cap, over seconds, 2.54 to 2.73 ms, 1730 to 1610); 2 x 1024 queries of
// 128 heads behind 7168 rows 2.08 to 2.14 ms; 2048 tokens of 128 heads 0.38 to 0.40 ms, 1420 to 1350.  A chunk
// took 2213 cycles (without the second sum) in the middle of a tile, a tile about 5500 more: the first
// softmax and the reading of the results, one after the other, and loads that wait for the stage that the
// results are in.  Tried without gain: the output freed in two halves, p . K of the last chunk before the
// next query is copied or in the order in which they are ready, 16-row steps of p . K left out where no
// row is seen.
#include <cmath>

#include "attend.cuh"
#include "device.cuh"
#include "launch.h"
#include "tensor.cuh"

namespace gkr {

namespace {

constexpr int kTileRows = 128;           // query heads of a tile, half of them in each CTA
constexpr int kCtaRows = 64;
constexpr int kChunk = 128;              // rows of K per chunk, half of them of each CTA
constexpr int kCtaKeys = 64;
constexpr int kStages = 3;
constexpr int kSoftmaxWarps = 8;         // warp w: tensor-memory lanes 32 (w % 4) .., half w / 4 of
                                         // their columns
constexpr int kMoveWarps = 8;            // write results, warp w of them as above
constexpr int kFirstMove = kSoftmaxWarps;
constexpr int kMmaWarp = kFirstMove + kMoveWarps;   // products (rank 0)
constexpr int kLoadWarp = kMmaWarp + 1;  // query tiles and rows for q . K; the pair's work
constexpr int kRefillWarp = kLoadWarp + 1;   // rows for p . K, the query's last dims
constexpr int kRelayWarp = kRefillWarp + 1;  // tells rank 0 what has landed
constexpr int kTileThreads = (kRelayWarp + 1) * 32;
constexpr uint32_t kBlockBytes = kCtaKeys * kRowBytes;      // 64 dims of 64 rows
constexpr uint32_t kHalfBytes = 4 * kBlockBytes;            // 256 dims
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr int kQTmemBlocks = 6;          // blocks of 64 dims of the query tile in tensor memory
constexpr uint32_t kQBytes = (8 - kQTmemBlocks) * kBlockBytes;   // and in shared memory
constexpr uint32_t kPBytes = 2 * kBlockBytes;               // probabilities of a chunk, bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;          // logits, 64 columns; output at 0
constexpr uint32_t kQCol = 320;          // the query's first 384 dims, two to a column
static_assert(kQCol + kQTmemBlocks * 32 == kTmemCols, "tensor memory");

// kind::f16 over the pair, M = 128, fp32 accumulator, bf16 A and B: logits N = 128, both K-major;
// output N = 256, B MN-major (bit 16).
constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
constexpr uint32_t kIdescS = idesc(kChunk, false);
constexpr uint32_t kIdescO = idesc(256, true);

// Shared memory of a CTA, from a 1024-byte boundary.
constexpr uint32_t kOffP = kQBytes;
constexpr uint32_t kOffStages = kOffP + kPBytes;
constexpr uint32_t kOffHeads = kOffStages + kStages * kStageBytes;   // [4][64] maxima, then sums, of a row
constexpr uint32_t kOffStats = kOffHeads + 256 * 4;         // [2][64] a tile's 1 / sum and log-sum-exp of a row
constexpr uint32_t kOffBars = kOffStats + 2 * 64 * 8;

// A pair takes its share of a tile in runs of at most so many chunks, each with an accumulator of its own, and joins
// them in fp32 rows in the workspace.  The tensor cores cut off what a sum of theirs cannot hold, all
// in one direction, on average half of its last bit for every 16 rows: in one run, results over a million rows
// came out 0.4 % too small, over 64 million 24 %; over 131072 it is 0.08 %, and a run costs what a tile does besides
// its chunks, 0.2 %.  That is a form of the kernel of its own (kLong), for calls with more rows than a run has, as
// the code that joins costs short calls 1 to 5 % (511 tokens of 16 heads 15.5 and 16.2 us, one query of each of 64
// requests over 4096 rows, 16 heads, 62.5 and 63.5).
constexpr int kRunChunks = 1024;

// A run of a pair's share of one tile, as its roles need it.
constexpr int kParts = 4;                // in the ring: the loads are never two tiles ahead
struct alignas(16) Part {
    int64_t row0;            // the tile's first row of q
    int64_t k0;              // the request's first row of K
    int64_t see;             // rows that the query of the tile's first row sees, not yet clamped
    int32_t offset;          // that row's head
    int32_t rows, keys;      // rows of the tile; rows of K
    int32_t least;           // rows that all of the tile's rows see
    int32_t chunks;          // of the tile; 0: no more parts
    int32_t from, to;        // of them, this pair's
    int32_t begin, end;      // and the run's
};

// Arguments of the tile kernel.
struct TileArgs {
    int32_t num_heads;
    uint32_t heads_shift;
    uint64_t heads_magic;        // x / num_heads = (x * heads_magic) >> heads_shift for x < 2^31
    int64_t num_tokens, num_rows;
    const int32_t* starts;       // null: one request, all queries and rows
    const int32_t* kv_starts;
    int32_t num_requests;
    int32_t causal;
    const int32_t* live;         // per row, < 0 or >= num_slots: no row; or null (one request only)
    int32_t num_slots;
    float sm_scale;
    void* out;                   // bf16 rows, or fp32 rows if `wide`
    float* lse;                  // natural, or in powers of two if `wide`
    int32_t wide;
    float* pieces;               // [pairs][2][slot_rows][512]
    float* piece_lse;            // [pairs][2][slot_rows]
    int4* meta;                  // [pairs] see kTailOpen
    int32_t slot_rows;           // rows of a piece at most
    int32_t* err;
};
// What a pair left in the workspace: slot 1, the beginning of a tile that the next pairs go on
// with (x: its first row, y: its rows); slot 0, a tile begun before, which it ended or not.
constexpr int kTailOpen = 1, kHeadThere = 2, kHeadEnds = 4;

// Work is counted in units of half a chunk; a tile costs kTileUnits besides its chunks (measured 5500
// cycles, a chunk 2213: with 2 units, 8192 x 64 heads took 2.64 ms instead of 2.31, as the pairs that
// have the short tiles at a prompt's beginning came last).
constexpr int kTileUnits = 4;
// Fewer units than this for each pair are not worth another piece to join (one query of 128 heads, 4096
// rows: 20.2 us, with 12 units 23.5).
constexpr int64_t kUnitsAPair = 6;
// To write pieces and join them takes as long as about so many units (511 tokens of 16 heads: whole
// tiles 17.3 us, cut 25.6; 200 of 32 13.8 and 18.2).
constexpr int64_t kJoinUnits = 8;
// No pair has a tile of its own where there are more units than this for each.
constexpr int64_t kWholeUnits = 64;

// A request: its queries, its rows of K.
struct Request {
    int32_t q0, queries, k0, keys;
    int32_t rows, tiles;     // of q
    __device__ __forceinline__ void derive(const TileArgs& p) {
        rows = queries * p.num_heads;
        tiles = static_cast<int32_t>((static_cast<uint32_t>(rows) + kTileRows - 1) / kTileRows);
    }
    __device__ __forceinline__ int64_t past() const { return static_cast<int64_t>(keys) - queries; }
};

__device__ __forceinline__ Request request_at(const TileArgs& p, int b, bool& bad) {
    const int32_t tokens = static_cast<int32_t>(p.num_tokens), rows = static_cast<int32_t>(p.num_rows);
    Request r;
    r.q0 = 0;
    r.k0 = 0;
    r.queries = tokens;
    r.keys = rows;
    if (p.starts != nullptr) {
        const int32_t a = p.starts[b], z = p.starts[b + 1], c = p.kv_starts[b], e = p.kv_starts[b + 1];
        r.q0 = min(max(a, 0), tokens);
        r.k0 = min(max(c, 0), rows);
        const int32_t q1 = min(max(z, r.q0), tokens), k1 = min(max(e, r.k0), rows);
        bad |= a != r.q0 || z != q1 || c != r.k0 || e != k1;
        r.queries = q1 - r.q0;
        r.keys = k1 - r.k0;
    }
    r.derive(p);
    return r;
}

// row / num_heads by a multiply and a shift (row < 2^31).
__device__ __forceinline__ int32_t query_of(const TileArgs& p, int32_t row) {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(row)) * p.heads_magic) >> p.heads_shift);
}
__device__ __forceinline__ int32_t clamped(int64_t see, int32_t keys) {
    return static_cast<int32_t>(min(max(see, INT64_C(0)), static_cast<int64_t>(keys)));
}
// How many rows row `row` of a request sees.
__device__ __forceinline__ int32_t sees(const TileArgs& p, const Request& r, int32_t row) {
    if (p.causal == 0) return r.keys;
    return clamped(r.past() + query_of(p, row) + 1, r.keys);
}
__device__ __forceinline__ int32_t chunks_in(int32_t keys) {
    return static_cast<int32_t>((static_cast<int64_t>(keys) + kChunk - 1) / kChunk);
}
// Chunks of a tile: what its last row sees.
__device__ __forceinline__ int32_t chunks_of(const TileArgs& p, const Request& r, int32_t tile) {
    return chunks_in(tile == r.tiles - 1 ? r.keys : sees(p, r, tile * kTileRows + kTileRows - 1));
}
// Units of the request's first `tile` tiles (tile < tiles).  Causal: tile x, but for the last,
// has max(0, ceil((past + floor((128 x + 127) / H) + 1) / 128)) chunks, which is
// max(0, floor((x + c) / H)) with c = floor((127 + (past + 128) H) / 128), as a tile and a chunk
// are both 128; and the sum of max(0, floor(y / H)) over y < z is H a (a - 1) / 2 + a (z - a H), a =
// floor(z / H).  (z < 2^31: the rows of K times H are at most 2^37.)
__device__ __forceinline__ int64_t floors_below(const TileArgs& p, int64_t z) {
    if (z <= 0) return 0;
    const int64_t a = query_of(p, static_cast<int32_t>(z));
    return p.num_heads * (a * (a - 1) / 2) + a * (z - a * p.num_heads);
}
__device__ __forceinline__ int64_t units_before(const TileArgs& p, const Request& r, int64_t tile) {
    if (p.causal == 0) return tile * (kTileUnits + 2 * chunks_in(r.keys));
    const int64_t c = (kTileRows - 1 + (r.past() + kChunk) * p.num_heads) >> 7;
    return kTileUnits * tile + 2 * (floors_below(p, tile + c) - floors_below(p, c));
}
__device__ __forceinline__ int64_t units_of(const TileArgs& p, const Request& r) {
    if (r.tiles == 0) return 0;
    return units_before(p, r, r.tiles - 1) + kTileUnits + 2 * chunks_in(r.keys);
}
// The chunk of a tile where a cut at this unit of it falls.
__device__ __forceinline__ int32_t chunk_at(int64_t unit) {
    return unit <= kTileUnits ? 0 : static_cast<int32_t>((unit - kTileUnits + 1) >> 1);
}

// A pair's parts, one after another.
struct Walk {
    Request r;
    int64_t left, unit;     // units left; units of the tile that are behind
    int32_t b, tile;
    // The one after `s` (at first one of no chunks); `chunks` 0 is a tile that sees no row here.
    template <bool kLong>
    __device__ bool next(const TileArgs& p, Part& s) {
        if (kLong && s.end < s.to) {
            s.begin = s.end;
            s.end = min(s.to, s.begin + kRunChunks);
            return true;
        }
        while (left > 0) {
            if (tile >= r.tiles) {
                if (++b >= p.num_requests) return false;
                bool bad = false;
                r = request_at(p, b, bad);
                tile = 0;
                unit = 0;
                continue;
            }
            const int32_t row = tile * kTileRows;
            s.row0 = static_cast<int64_t>(r.q0) * p.num_heads + row;
            s.k0 = r.k0;
            s.rows = min(kTileRows, r.rows - row);
            s.keys = r.keys;
            const int32_t query = query_of(p, row);
            s.offset = row - query * p.num_heads;
            s.see = p.causal == 0 ? r.keys : r.past() + query + 1;
            s.least = clamped(s.see, r.keys);
            s.chunks = chunks_of(p, r, tile);
            const int64_t all = kTileUnits + 2 * static_cast<int64_t>(s.chunks), first = unit;
            const int64_t take = min(left, all - unit);
            left -= take;
            unit += take;
            s.from = s.begin = chunk_at(first);
            s.to = chunk_at(unit);
            s.end = kLong ? min(s.to, s.begin + kRunChunks) : s.to;
            if (unit == all) {
                ++tile;
                unit = 0;
            }
            if (s.chunks == 0 ? first == 0 : s.to > s.from) return true;
        }
        return false;
    }
};

struct alignas(16) TileBarriers {
    // in the leader: arrivals of both CTAs
    uint64_t q_ready[2];           // relays: a query tile (even, odd) has landed
    uint64_t tail_ready;           // ... its last dims have
    uint64_t k_ready[2];           // all that q . K of a chunk (even, odd) waits for.  Relays: its rows
                                   // have landed; softmax: the logits before them are read
    uint64_t p_ready[2];           // and p . K.  Relays: its rows; softmax: the probabilities are written
    uint64_t o_free;               // movers: a tile's output is read
    // in each CTA
    uint64_t full[kStages];        // a query tile or rows for q . K have landed
    uint64_t refilled[kStages];    // rows for p . K have
    uint64_t tail;                 // the query's last dims have
    uint64_t empty[kStages];       // p . K of the chunk is complete; results have left the stage
    uint64_t s_full[2];            // the logits of a chunk are complete (even, odd chunks)
    uint64_t copied[2];            // a query tile is in tensor memory (even, odd tiles)
    uint64_t part[kParts];         // a part of the pair's work is described
    uint64_t stats[2];             // softmax: a tile's sums and log-sum-exps are there
    uint64_t drained;              // every product that was issued is complete
    int64_t sums[kTileThreads / 32];   // of the requests' units, if they are many
    uint32_t tmem_base;
    volatile int32_t timed_out;
    Part parts[kParts];
    Walk walk;                     // where the pair's work begins
};
constexpr size_t kTileSmem = kOffBars + sizeof(TileBarriers);
static_assert(kTileSmem <= 227 * 1024, "a CTA's shared memory");

// The requests' units are summed up by one warp, or, if there are many, first by all warps, each of
// them a run of requests per thread.
constexpr int kFewRequests = 64;
__device__ __forceinline__ int work_groups(const TileArgs& p) { return p.num_requests > kFewRequests ? kTileThreads / 32 : 1; }
__device__ __forceinline__ int64_t run_units(const TileArgs& p, int group, int lane, int& first, int& last, bool& bad) {
    const int run = (p.num_requests + 32 * work_groups(p) - 1) / (32 * work_groups(p));
    first = min(p.num_requests, (32 * group + lane) * run);
    last = min(p.num_requests, first + run);
    int64_t units = 0;
    for (int b = first; b < last; ++b) units += units_of(p, request_at(p, b, bad));
    return units;
}
__device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// A lane's value in an inclusive sum over the lanes.
template <typename T>
__device__ __forceinline__ T warp_upto(T v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(kFull, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// A pair's even share of the units, the first ones a unit more; false: none.
__device__ __forceinline__ bool even_share(int64_t total, int64_t pair, int64_t pairs, int64_t& x0, int64_t& units) {
    pairs = max(INT64_C(1), min(pairs, total / kUnitsAPair));
    const int64_t share = total >> 32 == 0 ? static_cast<uint32_t>(total) / static_cast<uint32_t>(pairs) : total / pairs;
    const int64_t more = total - share * pairs;
    x0 = pair * share + min(pair, more);
    units = pair >= pairs ? 0 : share + (pair < more ? 1 : 0);
    return units > 0;
}

// Where this pair's work begins and how much it is; a warp (sums: of the groups, if there are more
// than one).  Every instruction here is run for the first time and in a row, so what lanes have read
// is not read again.
__device__ __forceinline__ void find_work(const TileArgs& p, const int64_t* sums, int64_t pair, int64_t pairs, Walk& walk) {
    const int lane = threadIdx.x & 31, groups = work_groups(p);
    bool bad = false;
    walk.left = 0;
    walk.unit = 0;
    walk.b = p.num_requests;
    walk.tile = 0;
    Request mine_r = {};        // of the lane, where each has at most one
    int64_t before = 0, at;     // units before the group, then within a request
    int owner, b;
    if (p.num_requests <= 32) {
        int64_t mine = 0;
        int most = 0;
        if (lane < p.num_requests) {
            mine_r = request_at(p, lane, bad);
            mine = units_of(p, mine_r);
            if (mine_r.tiles > 0) most = kTileUnits + 2 * chunks_in(mine_r.keys);
        }
        const int64_t upto = warp_upto(mine, lane), total = __shfl_sync(kFull, upto, 31);
        bool whole = false;
        if (total <= pairs * kWholeUnits) {
            // Few tiles: one for each pair, if none of them takes much longer than an even share.
            const int tiles = warp_upto(mine_r.tiles, lane), all = __shfl_sync(kFull, tiles, 31);
            most = __reduce_max_sync(kFull, most);
            whole = all <= pairs &&
                    most <= static_cast<int>(static_cast<uint32_t>(total) / static_cast<uint32_t>(pairs)) + kJoinUnits;
            if (whole) {
                if (pair >= all) return;
                owner = __ffs(__ballot_sync(kFull, tiles > pair)) - 1;
                walk.tile = static_cast<int32_t>(pair) - __shfl_sync(kFull, tiles - mine_r.tiles, owner);
            }
        }
        if (!whole) {
            int64_t x0;
            if (!even_share(total, pair, pairs, x0, walk.left)) return;
            owner = __ffs(__ballot_sync(kFull, upto > x0)) - 1;
            at = x0 - __shfl_sync(kFull, upto - mine, owner);
        }
        walk.b = owner;
        walk.r.q0 = __shfl_sync(kFull, mine_r.q0, owner);
        walk.r.queries = __shfl_sync(kFull, mine_r.queries, owner);
        walk.r.k0 = __shfl_sync(kFull, mine_r.k0, owner);
        walk.r.keys = __shfl_sync(kFull, mine_r.keys, owner);
        walk.r.derive(p);
        if (whole) {
            walk.left = kTileUnits + 2 * static_cast<int64_t>(chunks_of(p, walk.r, walk.tile));
            return;
        }
    } else {
        int first = 0, last = 0;
        int64_t mine = groups == 1 ? run_units(p, 0, lane, first, last, bad) : lane < groups ? sums[lane] : 0;
        int64_t upto = warp_upto(mine, lane), x0;
        if (!even_share(__shfl_sync(kFull, upto, 31), pair, pairs, x0, walk.left)) return;
        if (groups > 1) {
            int g = 0;
            for (; g < groups - 1 && before + sums[g] <= x0; ++g) before += sums[g];
            mine = run_units(p, g, lane, first, last, bad);
            upto = warp_upto(mine, lane);
        }
        owner = __ffs(__ballot_sync(kFull, before + upto > x0)) - 1;
        at = x0 - before - (upto - mine);
        b = first;
        if (lane == owner) {
            for (; b < last - 1; ++b) {
                const int64_t u = units_of(p, request_at(p, b, bad));
                if (at < u) break;
                at -= u;
            }
        }
        walk.b = __shfl_sync(kFull, b, owner);
        at = __shfl_sync(kFull, at, owner);
        walk.r = request_at(p, walk.b, bad);
    }
    int64_t lo = 0, hi = walk.r.tiles;           // units_before(lo) <= at < units_before(hi)
#pragma unroll 1
    while (hi - lo > 1) {
        const int64_t x = lo + ((hi - lo) * lane >> 5);
        const uint32_t below = __ballot_sync(kFull, units_before(p, walk.r, x) <= at);   // lane 0 always
        const int n = __popc(below);
        const int64_t l = lo + ((hi - lo) * (n - 1) >> 5), h = n == 32 ? hi : lo + ((hi - lo) * n >> 5);
        lo = l;
        hi = h;
    }
    walk.tile = static_cast<int32_t>(lo);
    walk.unit = at - units_before(p, walk.r, lo);
}

// Values of key row `row` in this CTA's half of the dims (four blocks at `half`) that are not
// finite become 0; a warp.
__device__ __noinline__ void clear_row(uint32_t half, int row, int lane) {
    const uint32_t at = half + (lane >> 3) * kBlockBytes + row * kRowBytes + (lane & 7) * 16;
    uint4 v = lds16_at(at);
    uint32_t* const w = &v.x;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = w[i];
        const bool lo = (x & 0x7F80u) == 0x7F80u, hi = (x & 0x7F800000u) == 0x7F800000u;
        w[i] = (lo ? 0u : x & 0xFFFFu) | (hi ? 0u : x & 0xFFFF0000u);
        found |= lo || hi;
    }
    if (found) sts16(at, v);
}

// `rows` rows of 256 bytes from two swizzled blocks of 32 rows to global memory, `stride` bytes apart; a
// warp.
constexpr uint32_t kMoveBlock = 32 * kRowBytes;
__device__ __forceinline__ void copy_rows(uint32_t from, uint8_t* dst, int64_t stride, int rows, int lane) {
    const uint32_t block = from + (lane >> 3 & 1) * kMoveBlock;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        const uint4 x = lds16_at(block + r * kRowBytes + (((lane ^ r) & 7) << 4));
        if (r < rows) st16(dst + r * stride + 16 * (lane & 15), x);
    }
}

// Named barriers: the four softmax warps of each half of the rows; the movers.
constexpr int kHeadsBar = 1, kMoveBar = 3;

template <bool kLong>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
    tile_kernel(const TileArgs p, const __grid_constant__ CUtensorMap q_map,
                const __grid_constant__ CUtensorMap tail_map, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap out_map) {
    extern __shared__ __align__(1024) uint8_t smem[];
    TileBarriers* const bars = reinterpret_cast<TileBarriers*>(smem + kOffBars);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t pair = blockIdx.x >> 1;

    if (warp == kMmaWarp) {
        tmem_alloc_pair(smem_addr(&bars->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&bars->full[s]), 1);
            mbar_init(smem_addr(&bars->refilled[s]), 1);
            mbar_init(smem_addr(&bars->empty[s]), 1);
        }
        for (int s = 0; s < kParts; ++s) mbar_init(smem_addr(&bars->part[s]), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&bars->s_full[s]), 1);
            mbar_init(smem_addr(&bars->copied[s]), 1);
            mbar_init(smem_addr(&bars->stats[s]), kSoftmaxWarps);
            mbar_init(smem_addr(&bars->q_ready[s]), 2);
            mbar_init(smem_addr(&bars->k_ready[s]), 2 + 2 * kSoftmaxWarps);
            mbar_init(smem_addr(&bars->p_ready[s]), 2 + 2 * kSoftmaxWarps);
        }
        mbar_init(smem_addr(&bars->tail_ready), 2);
        mbar_init(smem_addr(&bars->tail), 1);
        mbar_init(smem_addr(&bars->o_free), 2 * kMoveWarps);
        mbar_init(smem_addr(&bars->drained), 1);
        bars->timed_out = 0;
        mbar_init_fence();
    }
    if (threadIdx.x == kLoadWarp * 32) {
        prefetch_map(&q_map);
        prefetch_map(&tail_map);
        prefetch_map(&k_map);
        prefetch_map(&out_map);
    }
    pdl_wait_previous();
    pdl_release_next();
    if (work_groups(p) > 1) {
        int first, last;
        bool bad = false;
        const int64_t units = warp_total(run_units(p, warp, lane, first, last, bad));
        if (lane == 0) bars->sums[warp] = units;
        if (bad && blockIdx.x == 0) report(p.err, kErrIndex);
    }
    if (work_groups(p) > 1) __syncthreads();
    Walk walk;
    if (warp == kLoadWarp) {
        find_work(p, bars->sums, pair, gridDim.x >> 1, walk);
        if (lane == 0) bars->walk = walk;
    }
    tc_fence_before_sync();
    __syncthreads();
    // The other CTA's barriers exist once both have come here; what only loads needs none of them.
    cluster_arrive();
    if (warp != kLoadWarp) cluster_wait();
    tc_fence_after_sync();
    // All 512 columns are this CTA's, so they begin at address 0.
    constexpr uint32_t tmem = 0;
    bool ok = bars->tmem_base == 0 && (smem_addr(smem) & 1023u) == 0u;
    // Part `tile` of the pair's work; a warp.  False after the last, or once a wait gave up.
    auto part_at = [&](int tile, Part& s) -> bool {
        if (!ok || !warp_wait(smem_addr(&bars->part[tile & (kParts - 1)]), (tile / kParts) & 1, ok)) return false;
        s = bars->parts[tile & (kParts - 1)];
        return s.chunks > 0;
    };
    // The last dims of a query tile; a thread.
    auto load_tail = [&](int64_t row0) {
        const uint32_t bar = smem_addr(&bars->tail);
        mbar_expect_tx(bar, kQBytes);
        tma_load_3d(smem_addr(smem), &tail_map, bar, 0, static_cast<int32_t>(row0 + rank * kCtaRows), kQTmemBlocks);
    };
    Ring<kStages> ring;

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------- rows for q . K
        // The warp walks through the pair's work and describes each part for the other roles; one
        // lane loads.  A part's description is replaced four parts on; as a tile's results keep
        // the stage of the next tile's query, the loads are never more than two tiles ahead of
        // the tile whose results are being written.
        int loads = 0, tile = 0;
        // the 64 rows from `row` on, all dims (a query's first 384): the next item of the ring
        auto load = [&](bool query, int64_t row) {
            if (loads >= kStages) warp_wait(smem_addr(&bars->empty[ring.s]), ring.parity ^ 1u, ok);
            if (!ok) return;
            if (lane == 0) {
                const uint32_t full = smem_addr(&bars->full[ring.s]);
                const uint32_t to = smem_addr(smem) + kOffStages + ring.s * kStageBytes;
                mbar_expect_tx(full, query ? kQTmemBlocks * kBlockBytes : kStageBytes);
                tma_load_3d(to, query ? &q_map : &k_map, full, 0, static_cast<int32_t>(row), 0);
                tma_load_3d(to + kHalfBytes, query ? &tail_map : &k_map, full, 0, static_cast<int32_t>(row), 4);
            }
            __syncwarp();
            ring.next();
            ++loads;
        };
        // The first tile's last dims come from here: they have landed before the refilling warp can ask
        // for the next ones.
        bool tail_asked = false;
        auto tail_landed = [&]() {
            if (tail_asked && !wait_landed(smem_addr(&bars->tail), 0)) ok = false;
            tail_asked = false;
        };
        Part s;
        s.end = s.to = 0;
        while (true) {
            const bool some = walk.next<kLong>(p, s);
            if (some && s.chunks == 0) {   // zeros, whatever has become of the other tiles
                const int rows = min(kCtaRows, s.rows - static_cast<int>(rank) * kCtaRows);
                const int64_t at = s.row0 + rank * kCtaRows, bytes = p.wide != 0 ? 2048 : 1024;
                for (int64_t i = lane * INT64_C(16); i < rows * bytes; i += 512)
                    st16(static_cast<uint8_t*>(p.out) + at * bytes + i, make_uint4(0u, 0u, 0u, 0u));
                for (int i = lane; i < rows; i += 32) p.lse[at + i] = -INFINITY;
                continue;
            }
            if (!ok) {
                if (!some) break;
                continue;
            }
            if (!some) s.chunks = 0;
            tail_landed();
            if (!ok) continue;
            if (lane == 0) {
                bars->parts[tile & (kParts - 1)] = s;
                mbar_arrive(smem_addr(&bars->part[tile & (kParts - 1)]));
            }
            __syncwarp();
            if (!some) break;
            if (++tile == 1) {
                if (lane == 0) load_tail(s.row0);
                tail_asked = true;
            }
            load(true, s.row0 + rank * kCtaRows);
#pragma unroll 1
            for (int c = s.begin; c < s.end && ok; ++c)
                load(false, s.k0 + static_cast<int64_t>(c) * kChunk + rank * kCtaKeys);
        }
        // what is under way lands before the CTA leaves
        tail_landed();
        for (int i = max(0, loads - kStages); i < loads; ++i)
            if (!wait_landed(smem_addr(&bars->full[i % kStages]), (i / kStages) & 1)) ok = false;
        __syncwarp();
        cluster_wait();
    } else if (warp == kRefillWarp) {
        // ------------------------------------------------------------- rows for p . K
        int j = 0, tile = 0, used[kStages] = {0, 0, 0};
        Part s;
        for (; part_at(tile, s); ++tile) {
            // q . K of the tile before is complete: the query's last dims may be replaced (the first
            // tile's come with the others)
            if (tile > 0 && lane == 0) load_tail(s.row0);
            __syncwarp();
            ring.next();   // the query tile
#pragma unroll 1
            for (int c = s.begin; c < s.end; ++c, ++j) {
                if (!warp_wait(smem_addr(&bars->s_full[j & 1]), (j >> 1) & 1, ok)) break;   // q . K has read it
                if (lane == 0) {
                    const uint32_t bar = smem_addr(&bars->refilled[ring.s]);
                    mbar_expect_tx(bar, kHalfBytes);
                    tma_load_3d(smem_addr(smem) + kOffStages + ring.s * kStageBytes + (1u - rank) * kHalfBytes, &k_map,
                                bar, 0,
                                static_cast<int32_t>(s.k0 + static_cast<int64_t>(c) * kChunk + (1u - rank) * kCtaKeys),
                                static_cast<int32_t>(4 * rank));
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kStages; ++i) used[i] += i == ring.s ? 1 : 0;
                ring.next();
            }
        }
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (used[i] > 0 && !wait_landed(smem_addr(&bars->refilled[i]), (used[i] - 1) & 1)) ok = false;
        if (tile > 1 && !wait_landed(smem_addr(&bars->tail), (tile - 1) & 1)) ok = false;
        __syncwarp();
    } else if (warp == kRelayWarp) {
        // ------------------------------------------------------------- what has landed
        // In the order in which the products need it.  No CTA's relay is a phase ahead of the other's: before
        // the next arrival at a barrier comes one that the products of the phase before must have
        // preceded (rows for p . K land after q . K).
        const uint32_t q_ready = map_rank(smem_addr(&bars->q_ready[0]), 0);
        const uint32_t tail_ready = map_rank(smem_addr(&bars->tail_ready), 0);
        const uint32_t k_ready = map_rank(smem_addr(&bars->k_ready[0]), 0);
        const uint32_t p_ready = map_rank(smem_addr(&bars->p_ready[0]), 0);
        uint32_t turns = 0;        // bit s: parity of the chunks that p has met in stage s
        int jq = 0, jo = 0;
        Ring<kStages> ro;          // the stage of chunk jo; `ring`: of the next item of the loads
        auto pass_on = [&](uint64_t* bar, uint32_t parity, uint32_t to) -> bool {
            if (!warp_wait(smem_addr(bar), parity, ok)) return false;
            if (lane == 0) mbar_arrive_cluster(to);
            return true;
        };
        auto refilled = [&]() -> bool {
            if (!pass_on(&bars->refilled[ro.s], turns >> ro.s & 1u, p_ready + 8 * (jo & 1))) return false;
            turns ^= 1u << ro.s;
            ro.next();
            ++jo;
            return true;
        };
        Part s;
        for (int tile = 0; part_at(tile, s); ++tile) {
            if (!pass_on(&bars->full[ring.s], ring.parity, q_ready + 8 * (tile & 1))) break;
            ring.next();
            if (tile > 0 && !refilled()) break;   // of the tile before
            ro = ring;
            if (!pass_on(&bars->tail, tile & 1, tail_ready)) break;
#pragma unroll 1
            for (int c = s.begin; c < s.end; ++c, ++jq) {
                if (!pass_on(&bars->full[ring.s], ring.parity, k_ready + 8 * (jq & 1))) break;
                ring.next();
                if (c > s.begin && !refilled()) break;
            }
            if (!ok) break;
        }
        if (ok && jo < jq) refilled();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------- products
        // The whole warp runs this, one lane issues (elect_lane).  q . K is one chunk ahead of p . K
        // within a tile; between tiles p . K of the last chunk comes first, as it and the writing of
        // the results take longer than what the next tile needs until its first p . K.
        if (rank == 0) {
            const uint32_t elected = elect_lane();
            const uint64_t q_desc = sw128_desc(smem_addr(smem));
            const uint64_t k_desc0 = sw128_desc(smem_addr(smem + kOffStages));
            const uint64_t v_desc0 = sw128_mn_desc(smem_addr(smem + kOffStages), kBlockBytes);
            const uint64_t p_desc0 = sw128_desc(smem_addr(smem + kOffP));
            const uint32_t q_lo = static_cast<uint32_t>(q_desc), k_lo = static_cast<uint32_t>(k_desc0);
            const uint32_t v_lo = static_cast<uint32_t>(v_desc0), p_lo = static_cast<uint32_t>(p_desc0);
            int jq = 0, jo = 0;                   // chunks multiplied by q, by p
            int tq = 0, to = 0, left_q = 0, left_next = 0, left_o = 0;   // parts begun, and what is left of them
            bool some = true, opened = false, fresh = true;   // opened: the next part's query is on its way
            Ring<kStages> rq;                     // the stage of chunk jq; `ring`: of chunk jo
            Part s;
#pragma unroll 1
            while (true) {
                if (some && left_q == 0 && !opened && jq - jo < 2) {
                    some = part_at(tq, s);
                    if (!ok) break;
                    if (!some) continue;
                    left_next = s.end - s.begin;
                    if (!warp_wait(smem_addr(&bars->q_ready[tq & 1]), (tq >> 1) & 1, ok)) break;
                    // q . K of the tile before has read its query
                    if (jq > 0 && !warp_wait(smem_addr(&bars->s_full[(jq - 1) & 1]), ((jq - 1) >> 1) & 1, ok)) break;
                    tc_fence_after_sync();
                    const uint32_t q = k_lo + rq.s * (kStageBytes >> 4);
                    if (elected) {
#pragma unroll 1
                        for (int b = 0; b < kQTmemBlocks; ++b)
#pragma unroll
                            for (int i = 0; i < 8; ++i)   // 8 dims
                                copy_to_tmem_pair(tmem + kQCol + 32 * b + 4 * i, desc_at(k_desc0, q + b * (kBlockBytes >> 4) + i));
                    }
                    __syncwarp();
                    mma_commit_pair(smem_addr(&bars->copied[tq & 1]), elected);
                    rq.next();
                    opened = true;
                } else if (some && jq - jo < 2 && !(opened && jo < jq)) {
                    if (opened) {
                        if (!warp_wait(smem_addr(&bars->tail_ready), tq & 1, ok)) break;
                        opened = false;
                        left_q = left_next;
                        ++tq;
                    }
                    if (!warp_wait(smem_addr(&bars->k_ready[jq & 1]), (jq >> 1) & 1, ok)) break;
                    tc_fence_after_sync();
                    const uint32_t b = k_lo + rq.s * (kStageBytes >> 4);
                    if (elected) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {       // 16 dims
                            const uint64_t bk = desc_at(k_desc0, b + (((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4));
                            if (k < 4 * kQTmemBlocks)
                                mma_bf16_ts_pair(tmem + kSCol, tmem + kQCol + 8 * k, bk, kIdescS, k != 0);
                            else
                                mma_bf16_ss_pair(tmem + kSCol,
                                                 desc_at(q_desc, q_lo + ((((k >> 2) - kQTmemBlocks) * kBlockBytes + (k & 3) * 32) >> 4)),
                                                 bk, kIdescS, true);
                        }
                    }
                    __syncwarp();
                    mma_commit_pair(smem_addr(&bars->s_full[jq & 1]), elected);
                    rq.next();
                    ++jq;
                    --left_q;
                } else if (jo < jq) {
                    if (left_o == 0) {
                        if (!part_at(to, s)) break;
                        left_o = s.end - s.begin;
                        ring.next();
                        ++to;
                        fresh = true;
                    }
                    if (!warp_wait(smem_addr(&bars->p_ready[jo & 1]), (jo >> 1) & 1, ok)) break;
                    if (fresh && to > 1 && !warp_wait(smem_addr(&bars->o_free), to & 1, ok)) break;   // of part to - 2
                    tc_fence_after_sync();
                    const uint32_t b = v_lo + ring.s * (kStageBytes >> 4);
                    if (elected) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {            // 16 rows; k / 4: of which CTA
#pragma unroll
                            for (int h = 0; h < 2; ++h)          // 128 of each CTA's 256 dims
                                mma_bf16_ss_pair(tmem + 128 * h, desc_at(p_desc0, p_lo + (((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4)),
                                                 desc_at(v_desc0, b + (((k >> 2) * kHalfBytes + (k & 3) * 2048 + h * 2 * kBlockBytes) >> 4)),
                                                 kIdescO, k != 0 || !fresh);
                        }
                    }
                    __syncwarp();
                    mma_commit_pair(smem_addr(&bars->empty[ring.s]), elected);
                    ring.next();
                    ++jo;
                    --left_o;
                    fresh = false;
                } else {
                    break;
                }
            }
            // whatever ended the loop, no product is under way when the pair leaves
            mma_commit_pair(smem_addr(&bars->drained), elected);
            if (!wait_landed(smem_addr(&bars->drained), 0)) ok = false;
            __syncwarp();
        }
    } else if (warp >= kFirstMove && warp < kMmaWarp) {
        // ------------------------------------------------------------- results
        // Warp w has tensor-memory lanes 32 (w % 4) .. and half w / 4 of what is in them: lane L is
        // row L % 64 of this CTA and of the output the dims 256 (L / 64) ...  The rows leave
        // through the stage of the next tile's query, once that is copied to tensor memory.
        const int quarter = warp & 3, part = (warp - kFirstMove) >> 2, half = quarter >> 1;
        const int row = (warp & 1) * 32 + lane;
        const int in_tile = static_cast<int>(rank) * kCtaRows + row;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t o_free = map_rank(smem_addr(&bars->o_free), 0);
        const bool first = threadIdx.x == kFirstMove * 32;
        if (first && rank == 0) p.meta[pair] = make_int4(0, 0, 0, 0);
        if (blockIdx.x == 0 && warp == kFirstMove && work_groups(p) == 1) {
            int from, upto;
            bool bad = false;
            run_units(p, 0, lane, from, upto, bad);
            if (bad) report(p.err, kErrIndex);
        }
        // Where run `s` goes: the results, or, where it does not end a whole tile, a piece (slot 1: of a share that
        // begins its tile; only the last one stays there).
        auto piece_of = [&](const Part& s) -> int64_t { return (2 * pair + (s.from == 0 ? 1 : 0)) * p.slot_rows; };
        auto whole_of = [&](const Part& s) -> bool { return s.from == 0 && s.end == s.chunks; };
        auto first_of = [&](const Part& s) -> int64_t { return whole_of(s) ? s.row0 : piece_of(s); };
        auto note = [&](const Part& s) {   // for the kernel that joins
            if (!first || rank != 0 || whole_of(s) || s.end < s.to) return;
            int4 mark = p.meta[pair];
            if (s.from != 0) {
                mark.z |= kHeadThere | (s.end == s.chunks ? kHeadEnds : 0);
            } else {
                mark.x = static_cast<int32_t>(s.row0);
                mark.y = s.rows;
                mark.z |= kTailOpen;
            }
            p.meta[pair] = mark;
        };
        auto set_lse = [&](const Part& s, float v) {
            if (half == 0 && part == 0 && in_tile < s.rows) (whole_of(s) ? p.lse : p.piece_lse)[first_of(s) + in_tile] = v;
        };
        Part s, n;
        int tile = 0;
        bool more = part_at(0, s);
        if (more) {
            // the first query's stage has no results to wait for
            if (warp_wait(smem_addr(&bars->copied[0]), 0, ok) && first) mbar_arrive(smem_addr(&bars->empty[0]));
            ring.next();
        }
        ok = !group_any(kMoveBar, kMoveWarps * 32, !ok);   // all movers leave together
#pragma unroll 1
        while (more && ok) {
            ring.skip(s.end - s.begin - 1);
            const Ring<kStages> last = ring;    // of the tile's chunks
            ring.next();                        // of the next query, if there is one
            more = part_at(tile + 1, n);
            if (more) warp_wait(smem_addr(&bars->copied[(tile + 1) & 1]), ((tile + 1) >> 1) & 1, ok);
            // The last value product implies everything before it.  The movers agree on it, so that
            // a row is written in full or not at all.
            if (ok) warp_wait(smem_addr(&bars->stats[tile & 1]), (tile >> 1) & 1, ok);
            if (ok) warp_wait(smem_addr(&bars->empty[last.s]), last.parity, ok);
            ok = !group_any(kMoveBar, kMoveWarps * 32, !ok);
            if (!ok) break;
            tc_fence_after_sync();
            float inv, lse2;
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(inv), "=f"(lse2)
                         : "r"(smem_addr(smem) + kOffStats + (tile & 1) * 512 + 8 * row) : "memory");
            // Each warp by itself: its 32 rows and 128 dims through 8 KB of the stage, in two blocks of
            // 128 bytes a row, swizzled.
            const uint32_t mine = smem_addr(smem) + kOffStages + ring.s * kStageBytes + (warp - kFirstMove) * 2 * kMoveBlock;
            const uint32_t to = mine + lane * kRowBytes + ((lane & 7) << 4);
            const int row0 = static_cast<int>(rank) * kCtaRows + (warp & 1) * 32;   // of the tile
            const int rows = min(s.rows - row0, 32);
            if ((!kLong || s.begin == s.from) && whole_of(s) && p.wide == 0) {
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {       // 64 dims, bf16
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float t[32];
                        tmem_ld32(tmem + lanes + 128 * part + 64 * b + 32 * h, t);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sts16((to ^ ((4 * h + i) << 4)) + b * kMoveBlock, pack8(t + 8 * i, inv));
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (rows == 32 && lane == 0) {
                        tma_store_3d(&out_map, mine + b * kMoveBlock, 0, static_cast<int32_t>(s.row0 + row0),
                                     4 * half + 2 * part + b);
                        bulk_commit();
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(o_free);
                if (rows < 32)   // the request's only
                    copy_rows(mine, static_cast<uint8_t*>(p.out) + (s.row0 + row0) * 1024 + (2 * half + part) * 256, 1024,
                              rows, lane);
            } else if (!kLong || s.begin == s.from) {
                uint8_t* const dst = (whole_of(s) ? static_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(p.pieces)) +
                                     (first_of(s) + row0) * 2048 + (2 * half + part) * 512;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {       // 64 dims, fp32
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float t[32];
                        tmem_ld32(tmem + lanes + 128 * part + 64 * b + 32 * h, t);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sts16((to ^ (i << 4)) + h * kMoveBlock, make_uint4(__float_as_uint(__fmul_rn(t[4 * i], inv)),
                                                                               __float_as_uint(__fmul_rn(t[4 * i + 1], inv)),
                                                                               __float_as_uint(__fmul_rn(t[4 * i + 2], inv)),
                                                                               __float_as_uint(__fmul_rn(t[4 * i + 3], inv))));
                    }
                    __syncwarp();
                    copy_rows(mine, dst + b * 256, 2048, rows, lane);
                    __syncwarp();   // read before it is written again
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(o_free);
            } else {
                // Joined with the share's runs before; each thread its row's 128 dims.
                const int64_t at = piece_of(s) + in_tile;
                const bool mine = in_tile < s.rows;
                const float old = mine ? p.piece_lse[at] : -INFINITY;
                const float top = fmaxf(old, lse2), ref = top == -INFINITY ? 0.0f : top;
                const float w_old = exp2_approx(__fsub_rn(old, ref)), w_new = exp2_approx(__fsub_rn(lse2, ref));
                const float sum = __fadd_rn(w_old, w_new), one = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
                lse2 = sum == 0.0f ? -INFINITY : __fadd_rn(top, log2f(sum));
                const int dim = 256 * half + 128 * part;
                float* const from = p.pieces + at * 512 + dim;
                uint8_t* const to_row = static_cast<uint8_t*>(p.out) + (s.row0 + in_tile) * (p.wide != 0 ? 2048 : 1024);
#pragma unroll 1
                for (int d = 0; d < 128; d += 16) {
                    float t[16];
                    tmem_ld16(tmem + lanes + 128 * part + d, t);
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 x = *reinterpret_cast<const float4*>(from + d + i);
                            const float o[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                t[i + k] = __fmul_rn(__fadd_rn(__fmul_rn(__fmul_rn(t[i + k], inv), w_new), __fmul_rn(o[k], w_old)), one);
                        }
                        if (whole_of(s) && p.wide == 0) {
                            st16(to_row + 2 * (dim + d), pack8(t));
                            st16(to_row + 2 * (dim + d) + 16, pack8(t + 8));
                        } else {
                            float* const to = whole_of(s) ? reinterpret_cast<float*>(to_row) + dim : from;
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<float4*>(to + d + i) = make_float4(t[i], t[i + 1], t[i + 2], t[i + 3]);
                        }
                    }
                    __syncwarp();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(o_free);
            }
            // what was read is read, before TMA writes there
            if (lane == 0) bulk_wait_read_all();
            fence_async_smem();
            group_sync(kMoveBar, kMoveWarps * 32);
            if (first && more) mbar_arrive(smem_addr(&bars->empty[ring.s]));
            set_lse(s, whole_of(s) && p.wide == 0 ? __fmul_rn(lse2, kLn2) : lse2);
            note(s);
            s = n;
            ++tile;
            ring.next();
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
        if (!ok) {
            // a wait gave up: what this pair has not written is marked
            walk = bars->walk;
            s.end = s.to = 0;
            for (int skip = tile; walk.next<kLong>(p, s);) {
                if (s.chunks == 0 || skip-- > 0) continue;
                set_lse(s, __uint_as_float(kUnwritten));
                note(s);
            }
        }
    } else {
        // ------------------------------------------------------------- softmax
        // Tensor-memory lane L: row L % 64 of this CTA; of a chunk the rows of CTA L / 64.  Two warps
        // share a lane, one for each half of its columns, so four threads have a row; they
        // exchange maxima and sums.
        const int quarter = warp & 3, part = warp >> 2;
        const int row = (warp & 1) * 32 + lane;
        const int half = quarter >> 1;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        float* const heads = reinterpret_cast<float*>(smem + kOffHeads) + row;
        const int self = (part * 2 + half) * 64;
        const uint32_t k_ready = map_rank(smem_addr(&bars->k_ready[0]), 0);
        const uint32_t p_ready = map_rank(smem_addr(&bars->p_ready[0]), 0);
        const float scale = __fmul_rn(p.sm_scale, kLog2e);   // logits in powers of two
        const uint32_t stages = smem_addr(smem) + kOffStages;
        // this thread's 64 bytes of the probabilities
        const uint32_t prow = smem_addr(smem) + kOffP + half * kBlockBytes + row * kRowBytes + ((part * 4 ^ (row & 7)) << 4);
        const int32_t column = half * kCtaKeys + part * 32;   // of the chunk
        auto head_sync = [&]() { group_sync(kHeadsBar + (warp & 1), 128); };
        auto head_any = [&](bool mine) -> bool { return group_any(kHeadsBar + (warp & 1), 128, mine); };
        uint32_t turns = 0;        // bit s: parity of the chunks so far in stage s
        int j = 0;
        if (lane == 0 && ok) mbar_arrive_cluster(k_ready);   // no logits before the first chunk's
        Ring<kStages> last;        // the stage of the chunk before
        Part s;
#pragma unroll 1
        for (int tile = 0;; ++tile) {
            const bool some = part_at(tile, s);
            ok = !head_any(!ok);       // a row's four warps leave together
            if (!ok || !some) break;
            ring.next();               // the query tile
            float m = -INFINITY, l = 0.0f, rounded = 0.0f;   // rounded: the sum of what p . K multiplies
            const int32_t in_tile = static_cast<int32_t>(rank) * kCtaRows + row;
            const int32_t see = p.causal == 0 ? s.keys
                                              : clamped(s.see + query_of(p, s.offset + in_tile), s.keys);
#pragma unroll 1
            for (int c = s.begin; c < s.end; ++c, ++j) {
                const bool fresh = c == s.begin;
                const int64_t key = static_cast<int64_t>(c) * kChunk + column;   // this thread's first
                uint32_t live = kFull;
                if (p.live != nullptr) {
                    const int32_t slot = key + lane < p.num_rows ? p.live[key + lane] : -1;
                    live = __ballot_sync(kFull, slot >= 0 && slot < p.num_slots);
                }
                if (ok) warp_wait(smem_addr(&bars->s_full[j & 1]), (j >> 1) & 1, ok);
                tc_fence_after_sync();
                float v[32];
                tmem_ld32(tmem + lanes + kSCol + 32 * part, v);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive_cluster(k_ready + 8 * ((j + 1) & 1));
                // columns that some row of the tile does not see
                if (key + 32 > s.least) {
                    const int64_t from = s.least - key;
                    uint32_t odd = 0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i >= from && !(fabsf(v[i]) <= 3.40282347e38f)) odd |= 1u << i;
                    odd = __reduce_or_sync(kFull, odd);
                    // A row of K with an infinity or a NaN makes every logit of its column one or
                    // the other, in both CTAs; other logits may be, and then nothing is cleared.
                    if (odd != 0u && ok && warp_wait(smem_addr(&bars->full[ring.s]), ring.parity, ok) &&
                        warp_wait(smem_addr(&bars->refilled[ring.s]), turns >> ring.s & 1u, ok)) {
                        for (uint32_t left = odd; left != 0u; left &= left - 1u)
                            clear_row(stages + ring.s * kStageBytes + half * kHalfBytes, part * 32 + __ffs(left) - 1, lane);
                    }
                    const int64_t lim = see - key;
                    live &= lim >= 32 ? kFull : lim <= 0 ? 0u : (1u << lim) - 1u;
                }
                const uint64_t scale2 = f32x2(scale, scale);
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    f32x2_split(mul_f32x2(f32x2(v[i], v[i + 1]), scale2), v[i], v[i + 1]);
                if (live != kFull) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (((live >> i) & 1u) == 0u) v[i] = -INFINITY;
                }
                float top = fmaxf(v[0], v[1]);
#pragma unroll
                for (int i = 2; i < 32; i += 2) top = fmaxf(top, fmaxf(v[i], v[i + 1]));
                // Rarely a logit is far above its row's reference; the row's four threads learn
                // of it by the barrier alone, and only then exchange their maxima.
                if (head_any(top > m + kLag || (m == -INFINITY && top > m))) {
                    heads[self] = top;
                    head_sync();
                    top = fmaxf(fmaxf(heads[0], heads[64]), fmaxf(heads[128], heads[192]));
                    head_sync();   // read before they are written again
                    const bool rise = top > m + kLag || (m == -INFINITY && top > m);
                    const float root = rise ? exp2_approx(__fmul_rn(__fsub_rn(m, top), 0.5f)) : 1.0f;
                    if (rise) m = top;
                    l = __fmul_rn(__fmul_rn(l, root), root);
                    rounded = __fmul_rn(__fmul_rn(rounded, root), root);
                    if (!fresh) {
                        // the products of the chunk before are in the accumulator
                        if (ok) warp_wait(smem_addr(&bars->empty[last.s]), last.parity, ok);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int d = 128 * part; d < 128 * part + 128 && ok; d += 32) {
                            float t[32];
                            tmem_ld32(tmem + lanes + d, t);
#pragma unroll
                            for (int i = 0; i < 32; ++i) t[i] = __fmul_rn(__fmul_rn(t[i], root), root);
                            tmem_st32(tmem + lanes + d, t);
                        }
                        tmem_st_wait();
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : __fsub_rn(m, kLift);
                const uint64_t ref2 = f32x2(-ref, -ref);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    f32x2_split(add_f32x2(f32x2(v[i], v[i + 1]), ref2), v[i], v[i + 1]);
                    v[i] = exp2_flush(v[i]);
                    v[i + 1] = exp2_flush(v[i + 1]);
                }
                uint64_t sum2 = add_f32x2(f32x2(v[0], v[1]), f32x2(v[2], v[3]));
#pragma unroll
                for (int i = 4; i < 32; i += 4)
                    sum2 = add_f32x2(sum2, add_f32x2(f32x2(v[i], v[i + 1]), f32x2(v[i + 2], v[i + 3])));
                float sum_a, sum_b;
                f32x2_split(sum2, sum_a, sum_b);
                l = __fadd_rn(l, __fadd_rn(sum_a, sum_b));
                // the chunk before is multiplied: its probabilities are read
                if (j > 0 && ok) warp_wait(smem_addr(&bars->empty[last.s]), last.parity, ok);
                uint4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack8(v + 8 * i);
                if (ok) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sts16(prow ^ (i << 4), w[i]);
                }
                fence_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive_cluster(p_ready + 8 * (j & 1));
                f32x2_split(add_f32x2(add_f32x2(sum_rounded(w[0]), sum_rounded(w[1])),
                                      add_f32x2(sum_rounded(w[2]), sum_rounded(w[3]))), sum_a, sum_b);
                rounded = __fadd_rn(rounded, __fadd_rn(sum_a, sum_b));
                last = ring;
                turns ^= 1u << ring.s;
                ring.next();
            }
            heads[self] = l;
            head_sync();
            const float total = __fadd_rn(__fadd_rn(heads[0], heads[64]), __fadd_rn(heads[128], heads[192]));
            head_sync();   // read before they are written again
            heads[self] = rounded;
            head_sync();
            const float divisor = __fadd_rn(__fadd_rn(heads[0], heads[64]), __fadd_rn(heads[128], heads[192]));
            head_sync();
            if (half == 0 && part == 0 && ok) {
                // both sums are 0 or neither is: what is not flushed is a normal bf16
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, divisor);
                const float lse2 = total == 0.0f ? -INFINITY : __fadd_rn(__fsub_rn(m, kLift), log2f(total));
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(smem_addr(smem) + kOffStats + (tile & 1) * 512 + 8 * row),
                             "f"(inv),
                             "f"(lse2) : "memory");
            }
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(smem_addr(&bars->stats[tile & 1]));
        }
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

// ---------------------------------------------------------------- pieces

// 16 dims of a row of fp32: four groups of four, 128 apart.
struct Dims {
    float4 d[4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __device__ __forceinline__ void add(const float* row, int lane, float w) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(row + 128 * i + 4 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i].x = __fmaf_rn(w, x[i].x, d[i].x);
            d[i].y = __fmaf_rn(w, x[i].y, d[i].y);
            d[i].z = __fmaf_rn(w, x[i].z, d[i].z);
            d[i].w = __fmaf_rn(w, x[i].w, d[i].w);
        }
    }
    __device__ __forceinline__ void store(uint8_t* row, int lane, float f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st8(row + 256 * i + 8 * lane, make_uint2(pack_bf16x2_rn(__fmul_rn(d[i].x, f), __fmul_rn(d[i].y, f)),
                                                     pack_bf16x2_rn(__fmul_rn(d[i].z, f), __fmul_rn(d[i].w, f))));
    }
};

// Joins the pieces of each tile that was cut, out = sum_i exp2(lse_i - lse) rows_i, and, where there are
// other results of the same rows (`own`), every row with those.  A block reads what the pairs left
// and goes through the rows that have something to join: a warp takes one, or, where there are few,
// two, four or eight warps, each of them some of the pieces.  (A block for each pair and eight rows,
// most of them with nothing to do, and one warp for up to 43 pieces took 20 us where this takes
// 6.)
constexpr int kJoinWarps = 8;
constexpr int32_t kMaxPairs = 128;
constexpr int kMaxParts = kMaxPairs + 1;    // of a row
struct JoinArgs {
    const float *own, *own_lse;       // fp32 rows, log-sum-exps in powers of two; or null
    const float *whole, *whole_lse;   // with `own`: the rows of the tiles that were not cut
    void* out;                        // bf16
    float* lse;
    int32_t pairs;
};
__global__ void __launch_bounds__(kJoinWarps * 32, 4) tile_join_kernel(const TileArgs p, const JoinArgs q) {
    // the cut tiles: first row, rows before (of cut tiles), pair that begins them; all pairs' flags
    __shared__ int32_t tail_row[kMaxPairs], tail_upto[kMaxPairs + 1], tail_pair[kMaxPairs], flags[kMaxPairs];
    __shared__ int32_t tails;
    __shared__ float weights[kJoinWarps][kMaxParts];
    __shared__ float4 parts[kJoinWarps][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_previous();
    pdl_release_next();
    if (warp == 0) {
        int n = 0, at = 0;
        if (lane == 0) tail_upto[0] = 0;
        int4 marks[kMaxPairs / 32];
#pragma unroll
        for (int i = 0; i < kMaxPairs / 32; ++i)
            marks[i] = 32 * i + lane < q.pairs ? p.meta[32 * i + lane] : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kMaxPairs / 32; ++i) {
            const int g = 32 * i + lane;
            const bool tail = (marks[i].z & kTailOpen) != 0;
            const uint32_t which = __ballot_sync(kFull, tail);
            const int upto = at + warp_upto(tail ? marks[i].y : 0, lane);
            const int k = n + __popc(which & ((1u << lane) - 1u));
            flags[g] = marks[i].z;
            if (tail) {
                tail_row[k] = marks[i].x;
                tail_pair[k] = g;
                tail_upto[k + 1] = upto;
            }
            n += __popc(which);
            at = __shfl_sync(kFull, upto, 31);
        }
        if (lane == 0) tails = n;
    }
    __syncthreads();
    const bool merge = q.own != nullptr;
    const int64_t total = merge ? p.num_tokens * p.num_heads : tail_upto[tails];
    // warps of a row, rows of a block at a time
    const int64_t blocks = gridDim.x;
    const int share = total <= blocks ? 8 : total <= 2 * blocks ? 4 : total <= 4 * blocks ? 2 : 1;
    const int each = kJoinWarps / share, sub = warp & (share - 1);
#pragma unroll 1
    for (int64_t base = blockIdx.x * static_cast<int64_t>(each); base < total; base += blocks * each) {
        const int64_t item = base + warp / share;
        const bool some = item < total;
        int64_t row = item;
        int g = 0, n = 0, r = 0;      // pair that begins the tile, pieces, row of the piece
        if (some && tails > 0) {
            const int32_t* const keys = merge ? tail_row : tail_upto;
            int lo = 0, hi = tails;   // the first of them past the item
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (keys[mid] <= item) lo = mid + 1;
                else hi = mid;
            }
            const int k = lo - 1;
            if (k >= 0) {
                r = static_cast<int>(item - keys[k]);
                if (r < tail_upto[k + 1] - tail_upto[k]) {
                    g = tail_pair[k];
                    row = tail_row[k] + static_cast<int64_t>(r);
                    // the pairs that go on with the tile, up to the one that ends it
                    n = 1;
                    while (g + n < q.pairs && (flags[g + n++] & kHeadEnds) == 0) {}
                }
            }
        }
        const int count = !some ? 0 : n + (merge ? 1 + (n == 0 ? 1 : 0) : 0);
        // part i of the row: a piece (the first ends its pair's run, slot 1, the others begin theirs, slot
        // 0) or the whole tile's row, then the other results'
        auto piece = [&](int i) -> int64_t { return (2 * static_cast<int64_t>(g + i) + (i == 0 ? 1 : 0)) * p.slot_rows + r; };
        auto row_of = [&](int i) -> const float* {
            return (i < n ? p.pieces + piece(i) * 512 : (i == count - 1 ? q.own : q.whole) + row * 512);
        };
        auto lse_of = [&](int i) -> float {
            return i < n ? p.piece_lse[piece(i)] : (i == count - 1 ? q.own_lse : q.whole_lse)[row];
        };
        float lses[(kMaxParts + 31) / 32], m = -INFINITY;
        bool unwritten = false;
#pragma unroll
        for (int i = 0; i < (kMaxParts + 31) / 32; ++i) {
            lses[i] = lane + 32 * i < count ? lse_of(lane + 32 * i) : -INFINITY;
            unwritten |= is_unwritten(lses[i]);
            m = fmaxf(m, lses[i]);
        }
        unwritten = __any_sync(kFull, unwritten) != 0;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
        const float ref = m == -INFINITY ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < (kMaxParts + 31) / 32; ++i) {
            const float w = exp2_approx(__fsub_rn(lses[i], ref));
            if (lane + 32 * i < count) weights[warp][lane + 32 * i] = w;
            sum = __fadd_rn(sum, w);
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, x));
        __syncwarp();
        Dims acc;
        acc.zero();
#pragma unroll 4
        for (int i = sub; i < count; i += share) acc.add(row_of(i), lane, weights[warp][i]);
        if (share > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) parts[warp][32 * i + lane] = acc.d[i];
            __syncthreads();
            if (sub == 0)
                for (int w = 1; w < share; ++w) acc.add(reinterpret_cast<const float*>(parts[warp + w]), lane, 1.0f);
            __syncthreads();
        }
        if (some && sub == 0) {
            if (!unwritten) {
                acc.store(static_cast<uint8_t*>(q.out) + row * 1024, lane, sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum));
                if (lane == 0) q.lse[row] = sum == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, log2f(sum)), kLn2);
            } else if (lane == 0) {
                q.lse[row] = __uint_as_float(kUnwritten);
            }
        }
        __syncwarp();   // the weights are read before the next row's are written
    }
}

// ---------------------------------------------------------------- host

// `rows` rows of 512 bf16 (`stride` bytes apart) as a 3-D tensor map of 64 dims x rows x 8 blocks of
// dims, with boxes of `box_rows` rows of `blocks` blocks: one load brings those dims of the rows as so many
// operand blocks.  Rows past the last read as zeros.
cudaError_t rows_tensor_map(const void* base, int64_t rows, int64_t stride, uint32_t box_rows, uint32_t blocks,
                            CUtensorMap* map) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), 8};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride), 128};
    const cuuint32_t box[3] = {64, box_rows, blocks};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r =
        encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The workspace of a tile launch: pieces, their log-sum-exps, what each pair left.
constexpr int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
int32_t slot_rows(int64_t rows) { return static_cast<int32_t>(rows < kTileRows ? rows : kTileRows); }
int64_t tile_bytes(int32_t pairs, int64_t rows) {
    const int64_t n = 2 * static_cast<int64_t>(pairs) * slot_rows(rows);
    return n * 2048 + up16(n * 4) + static_cast<int64_t>(pairs) * 16;
}

cudaError_t tile_pairs(int32_t* pairs) {
    const cudaError_t e = resident_pairs(reinterpret_cast<const void*>(tile_kernel<false>), kTileThreads, kTileSmem, pairs);
    if (*pairs > kMaxPairs) *pairs = kMaxPairs;
    return e;
}

// Attention of the rows of q; args but for what is in the workspace.  Joined with other results, if
// there are any (own; then the tiles leave fp32 rows).
cudaError_t launch_tiles(TileArgs a, JoinArgs join, const void* q, const void* kv, int64_t kv_stride, uint8_t* workspace,
                         int32_t pdl, cudaStream_t stream) {
    int32_t pairs = 0;
    cudaError_t e = tile_pairs(&pairs);
    if (e != cudaSuccess) return e;
    // ceil(2^shift / d) with shift = 32 + ceil(log2(d)): the product's excess over x 2^shift / d is below
    // 2^31 < 2^shift / d
    a.heads_shift = 32;
    while ((1 << (a.heads_shift - 32)) < a.num_heads) ++a.heads_shift;
    a.heads_magic = ((UINT64_C(1) << a.heads_shift) + a.num_heads - 1) / a.num_heads;
    const int64_t rows = a.num_tokens * a.num_heads;
    a.slot_rows = slot_rows(rows);
    const int64_t n = 2 * static_cast<int64_t>(pairs) * a.slot_rows;
    a.pieces = reinterpret_cast<float*>(workspace);
    a.piece_lse = reinterpret_cast<float*>(workspace + n * 2048);
    a.meta = reinterpret_cast<int4*>(workspace + n * 2048 + up16(n * 4));
    CUtensorMap q_map, tail_map, k_map, out_map;
    // no rows: nothing is loaded by their map; fp32 results do not leave by theirs
    e = rows_tensor_map(q, rows, 1024, kCtaRows, 4, &q_map);
    if (e == cudaSuccess) e = rows_tensor_map(q, rows, 1024, kCtaRows, 8 - kQTmemBlocks, &tail_map);
    if (e == cudaSuccess)
        e = a.num_rows > 0 ? rows_tensor_map(kv, a.num_rows, kv_stride * 2, kCtaKeys, 4, &k_map)
                           : rows_tensor_map(q, rows, 1024, kCtaRows, 4, &k_map);
    if (e == cudaSuccess) e = rows_tensor_map(a.out, rows, 1024, 32, 1, &out_map);
    if (e != cudaSuccess) return e;
    const bool longer = a.num_rows > static_cast<int64_t>(kRunChunks) * kChunk;   // some tile's share may take runs
    if (longer) {   // the kernel's limit of shared memory is set with this
        int32_t same = 0;
        e = resident_pairs(reinterpret_cast<const void*>(tile_kernel<true>), kTileThreads, kTileSmem, &same);
        if (e != cudaSuccess) return e;
    }
    e = launch_kernel(longer ? tile_kernel<true> : tile_kernel<false>, 2 * static_cast<int64_t>(pairs), kTileThreads,
                      kTileSmem, stream, pdl, a, q_map, tail_map, k_map, out_map);
    if (e != cudaSuccess) return e;
    // a block for each row that may have something to join, up to one wave
    int64_t warps = 0;
    e = resident_warps(reinterpret_cast<const void*>(tile_join_kernel), kJoinWarps * 32, 0, &warps);
    if (e != cudaSuccess) return e;
    const int64_t most = join.own != nullptr ? rows : static_cast<int64_t>(pairs) * a.slot_rows;
    const int64_t wave = warps / kJoinWarps, blocks = most < wave ? most : wave;
    join.pairs = pairs;
    return launch_kernel(tile_join_kernel, blocks, kJoinWarps * 32, 0, stream, pdl, a, join);
}

// The workspace of a prefix attention: the prefix as bf16 rows, both parts' rows and
// log-sum-exps, both parts' own workspaces.
struct PrefixLayout {
    bool written_out;    // every query's list with the prefix in front of it
    int64_t rows, shared, shared_lse, own, own_lse, tiles, attend, bytes;
};
// Two ways: the prefix once for all queries (gathered, tiles of 128 query heads, the queries' own
// lists, the join: five launches), or, as the sparse attention does, each query's list with the
// prefix in front of it (two launches, 128 rows of the tensor cores for a query's heads, every record
// dequantised for every query).  Which takes less by these estimates, in us:
//   written out: 10.5 and 1.05 for a chunk of 64 records of a pair's run;
//   shared: 27, the gather 2.1e-4 a record, 1.35 for a chunk of 128 rows of a pair's run and
//   1.05 for one of 64 own records.
// Measured, us in a graph, shared and written out (queries x heads, prefix + 100 own): 4 x 16, 4095 30.0
// and 16.0, 16384 37.2 and 26.8, 65536 57 and 68; 16 x 16, 4095 31.5 and 30.1, 16384 38 and 72; 64 x 16,
// 2048 33 and 42, 131072 205 and 1801; 16 x 128, 16384 67 and 77; 64 x 64, 2048 43.7 and 42.8; 128 x 64,
// 512 43.5 and 31.8, 4095 83 and 140.  Of 90 sizes (1 to 128 queries, 16, 64, 128 heads, 512 to 131072
// records) the slower way is taken in two: 64 x 64, 2048, by 2 %, and 128 x 128, 2048, by 21 % (98 and 81), as the
// estimates leave out what the fp32 rows of many heads and their join take.
bool write_out(int32_t num_heads, int64_t num_queries, int64_t prefix_length, int64_t topk, int32_t pairs) {
    const double own = static_cast<double>(num_queries) * static_cast<double>((topk + 63) / 64) / pairs;
    const double listed = static_cast<double>(num_queries) * static_cast<double>((prefix_length + topk + 63) / 64) / pairs;
    const double tiles = static_cast<double>((num_queries * num_heads + kTileRows - 1) / kTileRows);
    const double shared = tiles * static_cast<double>((prefix_length + kChunk - 1) / kChunk) / pairs;
    return 10.5 + 1.05 * listed <= 27.0 + 2.1e-4 * static_cast<double>(prefix_length) + 1.35 * shared + 1.05 * own;
}
cudaError_t prefix_layout(int32_t num_heads, int64_t num_queries, int64_t prefix_length, int64_t topk,
                          PrefixLayout* w) {
    const int64_t n = num_queries * num_heads;
    *w = {};
    int32_t pairs = 0;
    cudaError_t e = tile_pairs(&pairs);
    if (e != cudaSuccess) return e;
    w->written_out = write_out(num_heads, num_queries, prefix_length, topk, pairs);
    if (w->written_out) return attention_workspace(num_heads, num_queries, prefix_length + topk, &w->bytes);
    const bool both = prefix_length > 0 && topk > 0;
    int64_t at = 0, attend = 0;
    if (topk > 0) e = attention_workspace(num_heads, num_queries, topk, &attend);
    if (e != cudaSuccess) return e;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 127) / 128 * 128;
        return here;
    };
    w->rows = take(prefix_length * 1024);
    w->shared = take(both ? n * 2048 : 0);
    w->shared_lse = take(both ? n * 4 : 0);
    w->own = take(both ? n * 2048 : 0);
    w->own_lse = take(both ? n * 4 : 0);
    w->tiles = take(tile_bytes(pairs, n));
    w->attend = take(attend);
    w->bytes = at;
    return cudaSuccess;
}

}  // namespace

cudaError_t prompt_workspace(int32_t num_heads, int64_t num_tokens, int64_t* bytes) {
    int32_t pairs = 0;
    const cudaError_t e = tile_pairs(&pairs);
    if (e != cudaSuccess) return e;
    *bytes = tile_bytes(pairs, num_tokens * num_heads);
    return cudaSuccess;
}

cudaError_t prefix_workspace(int32_t num_heads, int64_t num_queries, int64_t prefix_length, int64_t topk,
                             int64_t* bytes) {
    PrefixLayout w;
    const cudaError_t e = prefix_layout(num_heads, num_queries, prefix_length, topk, &w);
    *bytes = e == cudaSuccess ? w.bytes : 0;
    return e;
}

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t stream) {
    TileArgs a = {};
    a.num_heads = p.num_heads;
    a.num_tokens = p.num_tokens;
    a.num_rows = p.num_rows;
    a.starts = p.starts;
    a.kv_starts = p.kv_starts;
    a.num_requests = p.num_requests;
    a.causal = p.causal;
    a.sm_scale = p.sm_scale;
    a.out = p.out;
    a.lse = p.lse;
    a.err = p.err;
    JoinArgs join = {};
    join.out = p.out;
    join.lse = p.lse;
    return launch_tiles(a, join, p.q, p.kv, p.kv_stride, static_cast<uint8_t*>(p.workspace), p.pdl, stream);
}

cudaError_t launch_prefix_attention(const PrefixParams& p, cudaStream_t stream) {
    const AttentionParams& o = p.own;
    PrefixLayout w;
    cudaError_t e = prefix_layout(o.num_heads, o.num_queries, p.prefix_length, o.topk, &w);
    if (e != cudaSuccess) return e;
    uint8_t* const base = static_cast<uint8_t*>(o.workspace);
    const bool both = p.prefix_length > 0 && o.topk > 0;
    AttentionParams own = o;
    own.parted = 1;
    own.workspace = base + w.attend;
    if (w.written_out) {
        own.prefix = p.prefix;
        own.prefix_length = p.prefix_length;
        own.topk += p.prefix_length;
        return launch_sparse_attention(own, stream);
    }
    if (both) {
        own.out = base + w.own;
        own.lse = reinterpret_cast<float*>(base + w.own_lse);
        own.wide = 1;
        e = launch_sparse_attention(own, stream);
        if (e != cudaSuccess) return e;
    }
    GatherParams g = {};
    g.cache = o.cache;
    g.page_stride = o.page_stride;
    g.block_size = o.block_size;
    g.num_slots = o.num_slots;
    g.indices = p.prefix;
    g.num_indices = p.prefix_length;
    g.out = base + w.rows;
    g.err = o.err;
    g.pdl = o.pdl;
    e = launch_gather_mxfp4(g, stream);
    if (e != cudaSuccess) return e;
    TileArgs a = {};
    a.num_heads = o.num_heads;
    a.num_tokens = o.num_queries;
    a.num_rows = p.prefix_length;
    a.num_requests = 1;
    a.live = p.prefix;
    a.num_slots = o.num_slots;
    a.sm_scale = o.sm_scale;
    a.out = both ? static_cast<void*>(base + w.shared) : o.out;
    a.lse = both ? reinterpret_cast<float*>(base + w.shared_lse) : o.lse;
    a.wide = both ? 1 : 0;
    a.err = o.err;
    JoinArgs join = {};
    join.out = o.out;
    join.lse = o.lse;
    if (both) {
        join.own = reinterpret_cast<const float*>(base + w.own);
        join.own_lse = reinterpret_cast<const float*>(base + w.own_lse);
        join.whole = reinterpret_cast<const float*>(base + w.shared);
        join.whole_lse = reinterpret_cast<const float*>(base + w.shared_lse);
    }
    return launch_tiles(a, join, o.q, base + w.rows, 512, base + w.tiles, o.pdl, stream);
}

}  // namespace gkr
