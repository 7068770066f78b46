// Host side of the C ABI declared in include/gkr.h: argument checks, geometry
// and kernel dispatch.  No allocation, no synchronisation, no exceptions.
#include "gkr.h"
#include "launch.h"

#include <atomic>
#include <cstdint>
#include <mutex>
#include <vector>

namespace {

thread_local int32_t g_last_cuda_error = 0;
std::atomic<int> g_pdl{1};
std::atomic<int> g_early_metadata{0};
constexpr int64_t kDefaultStagedMin = 24576;
constexpr int64_t kDefaultStreamMin = 131072;
constexpr int64_t kMaxRows = INT64_C(1) << 24;   // queries, list entries of a call at most
constexpr int64_t kMaxList = INT64_C(1) << 21;   // entries of an eviction list at most
constexpr int64_t kMaxIndex = INT64_C(0x7FFFFFFF);
constexpr int64_t kMaxPromptRows = INT64_C(0x7FFF0000);   // rows of a prompt attention at most
constexpr int32_t kMaxQHeads = 4096;   // query heads per token (padded) at most
std::atomic<int64_t> g_staged_min{kDefaultStagedMin};
std::atomic<int64_t> g_stream_min{kDefaultStreamMin};

struct OccEntry {
    int device;
    const void* func;
    size_t smem;
    int threads;
    int64_t warps;
};
std::mutex g_occ_mutex;
std::vector<OccEntry> g_occ;

struct PairEntry {
    int device;
    const void* func;
    int32_t pairs;
};
std::vector<PairEntry> g_pairs;

struct RecordRows {
    int32_t data, scale, align;
};

bool record_rows(int32_t record, RecordRows* r) {
    // V4.1: 512 B e4m3 + 16 UE8M0; V4: 448 B e4m3 + 128 B bf16 + 7 UE8M0 + 1 pad.
    // Pages align to 512 B (V4.1) and 576 B (V4) ("PR #56893 [DSv4.1] Store the whole
    // KV in MXFP8 (FlashMLA V4.1 record)", section "功能与动机").  The plain KV-only
    // caches keep 512 elements a row: fp8 e4m3 (512 B) or bf16 (1024 B), pages aligned
    // to 512 B ("PR #56441 [Perf][DSpark] KV-only context insertion across V4.1 cache
    // formats", section "实现拆解" item 1).
    // MXFP4 (the library's own record): 256 B e2m1 + 16 UE8M0, pages aligned to 512 B.
    if (record == 272) { *r = {256, 16, 512}; return true; }
    if (record == 528) { *r = {512, 16, 512}; return true; }
    if (record == 584) { *r = {576, 8, 576}; return true; }
    if (record == 512) { *r = {512, 0, 512}; return true; }
    if (record == 1024) { *r = {1024, 0, 512}; return true; }
    return false;
}

bool packed(int32_t record) { return record == 528 || record == 584 || record == 272; }
// The records of the pages' compressed writer.
bool compressed(int32_t record) { return record == 528 || record == 584; }

// Packed records need block_size % 32 == 0 (the page geometry of the pages); the
// plain caches take any block_size >= 1.
bool block_size_ok(int32_t record, int32_t bs) {
    return bs > 0 && (!packed(record) || bs % 32 == 0);
}

// Query heads and rows of a prompt attention: tiles of rows are addressed in 32 bits.
bool prompt_rows_ok(int32_t num_heads, int64_t num_tokens) {
    return num_heads >= 1 && num_heads <= kMaxQHeads && num_tokens >= 0 &&
           num_tokens <= kMaxPromptRows / num_heads;
}
bool prefix_sizes_ok(int32_t num_heads, int64_t num_queries, int64_t prefix_length, int64_t topk) {
    return num_heads >= 1 && num_heads <= gkr::kAttentionMaxHeads && num_queries >= 0 &&
           num_queries <= kMaxRows && prefix_length >= 0 && prefix_length <= kMaxRows && topk >= 0 &&
           topk <= kMaxRows && prompt_rows_ok(num_heads, num_queries) &&
           num_queries * ((topk + 63) / 64) <= kMaxIndex;
}

bool finite(float x) { return x >= -3.40282347e38f && x <= 3.40282347e38f; }

// Whether two ranges of bytes have one in common.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

gkr_status check_cache(const gkr_cache_desc* c, RecordRows* rows) {
    if (c == nullptr) return GKR_EINVAL;
    if (!record_rows(c->record, rows)) return GKR_EUNSUPPORTED_RECORD;
    if (!block_size_ok(c->record, c->block_size)) return GKR_EINVAL;
    if (c->num_pages <= 0) return GKR_EINVAL;
    if (c->num_pages > (INT64_C(0x7FFFFFFF) / c->block_size)) return GKR_EINVAL;  // slots < 2^31
    const int64_t need = static_cast<int64_t>(c->block_size) * c->record;
    if (need > INT64_C(0x7FFFFFFF)) return GKR_EINVAL;                             // page < 2^31 B
    if (c->page_stride < need || c->page_stride % rows->align != 0) return GKR_EBAD_PAGE_GEOMETRY;
    if (c->page_stride > INT64_MAX / c->num_pages) return GKR_EBAD_PAGE_GEOMETRY;
    return GKR_OK;
}

gkr_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return GKR_OK;
    g_last_cuda_error = static_cast<int32_t>(e);
    return GKR_ECUDA;
}

// The launch policy of one call: the process-wide defaults (gkr_set_*), overridden by
// the fields of `o` that are not -1.  GKR_EINVAL for any other negative value, or a
// flag other than -1, 0 or 1.
struct Policy {
    int32_t pdl, early_metadata;
    int64_t staged_min, stream_min;
};

gkr_status resolve_policy(const gkr_launch_opts* o, Policy* out) {
    out->pdl = g_pdl.load(std::memory_order_relaxed);
    out->early_metadata = g_early_metadata.load(std::memory_order_relaxed);
    out->staged_min = g_staged_min.load(std::memory_order_relaxed);
    out->stream_min = g_stream_min.load(std::memory_order_relaxed);
    if (o == nullptr) return GKR_OK;
    if (o->pdl < -1 || o->pdl > 1 || o->early_metadata < -1 || o->early_metadata > 1 ||
        o->insert_staged_min < -1 || o->insert_stream_min < -1)
        return GKR_EINVAL;
    if (o->pdl >= 0) out->pdl = o->pdl;
    if (o->early_metadata >= 0) out->early_metadata = o->early_metadata;
    if (o->insert_staged_min >= 0) out->staged_min = o->insert_staged_min;
    if (o->insert_stream_min >= 0) out->stream_min = o->insert_stream_min;
    return GKR_OK;
}

}  // namespace

namespace gkr {

cudaError_t resident_warps(const void* func, int threads, size_t smem, int64_t* warps) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_occ_mutex);
    for (const OccEntry& o : g_occ) {
        if (o.device == dev && o.func == func && o.smem == smem && o.threads == threads) {
            *warps = o.warps;
            return cudaSuccess;
        }
    }
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, func, threads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    const int64_t w = static_cast<int64_t>(sms) * per_sm * (threads / 32);
    try {
        g_occ.push_back({dev, func, smem, threads, w});
    } catch (...) {   // asked again next time
    }
    *warps = w;
    return cudaSuccess;
}

cudaError_t resident_pairs(const void* func, int threads, size_t smem, int32_t* pairs) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_occ_mutex);
    for (const PairEntry& o : g_pairs) {
        if (o.device == dev && o.func == func) {
            *pairs = o.pairs;
            return cudaSuccess;
        }
    }
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, func, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    try {
        g_pairs.push_back({dev, func, n});
    } catch (...) {   // asked again next time
    }
    *pairs = n;
    return cudaSuccess;
}

}  // namespace gkr

extern "C" {

GKR_API void gkr_set_pdl(int32_t enable) { g_pdl.store(enable ? 1 : 0); }

GKR_API int32_t gkr_get_pdl(void) { return g_pdl.load() ? 1 : 0; }

GKR_API void gkr_set_early_metadata(int32_t enable) { g_early_metadata.store(enable ? 1 : 0); }

GKR_API int32_t gkr_get_early_metadata(void) { return g_early_metadata.load() ? 1 : 0; }

GKR_API void gkr_set_insert_stream_min(int64_t tokens) {
    g_stream_min.store(tokens < 0 ? kDefaultStreamMin : tokens);
}

GKR_API int64_t gkr_get_insert_stream_min(void) { return g_stream_min.load(); }

GKR_API void gkr_set_insert_staged_min(int64_t tokens) {
    g_staged_min.store(tokens < 0 ? kDefaultStagedMin : tokens);
}

GKR_API int64_t gkr_get_insert_staged_min(void) { return g_staged_min.load(); }

GKR_API int64_t gkr_page_stride(int32_t record, int32_t block_size) {
    RecordRows r;
    if (!record_rows(record, &r) || !block_size_ok(record, block_size)) return -1;
    const int64_t need = static_cast<int64_t>(block_size) * record;
    return (need + r.align - 1) / r.align * r.align;
}

GKR_API gkr_status gkr_record_rows(int32_t record, int32_t* data_row_bytes,
                                   int32_t* scale_row_bytes, int32_t* page_align) {
    RecordRows r;
    if (!record_rows(record, &r)) return GKR_EUNSUPPORTED_RECORD;
    if (data_row_bytes) *data_row_bytes = r.data;
    if (scale_row_bytes) *scale_row_bytes = r.scale;
    if (page_align) *page_align = r.align;
    return GKR_OK;
}

}  // extern "C"

namespace {

// Checks shared by the insert entry points; fills `p` on success.  A GKR_OK status
// with p.num_tokens == 0 means there is nothing to launch.
gkr_status prepare_insert(const void* kv, int64_t num_tokens, void* k_cache,
                          const gkr_cache_desc* cache, const int64_t* slot_mapping,
                          const int64_t* positions, const float* cos_sin_cache, int64_t max_pos,
                          const float* fp8_scale, int32_t* err_flag,
                          const gkr_launch_opts* opts, gkr::InsertParams* p) {
    RecordRows rows;
    gkr_status st = check_cache(cache, &rows);
    if (st != GKR_OK) return st;
    Policy pol;
    st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (num_tokens < 0) return GKR_EINVAL;
    p->num_tokens = num_tokens;
    if (num_tokens == 0) return GKR_OK;  // the descriptor is checked; nothing else is read
    if (max_pos <= 0 || max_pos > INT64_C(0x7FFFFFFF)) return GKR_EINVAL;
    if (!kv || !k_cache || !slot_mapping || !positions || !cos_sin_cache) return GKR_EINVAL;
    const bool fp8 = cache->record == 512;  // fp8_scale is read for fp8 rows only
    if (fp8 && !fp8_scale) return GKR_EINVAL;
    if (!aligned(kv, 16) || !aligned(k_cache, 16) || !aligned(cos_sin_cache, 16) ||
        !aligned(slot_mapping, 8) || !aligned(positions, 8) || !aligned(err_flag, 4) ||
        (fp8 && !aligned(fp8_scale, 4)))
        return GKR_EALIGN;
    p->kv = kv;
    p->cache = static_cast<uint8_t*>(k_cache);
    p->page_stride = cache->page_stride;
    p->block_size = cache->block_size;
    p->num_slots = static_cast<int32_t>(cache->num_pages * cache->block_size);
    p->slots = slot_mapping;
    p->positions = positions;
    p->csc = cos_sin_cache;
    p->max_pos = max_pos;
    p->ratio = 1;
    p->fp8_scale = cache->record == 512 ? fp8_scale : nullptr;
    p->err = err_flag;
    p->early_metadata = pol.early_metadata;
    p->pdl = pol.pdl;
    p->staged_min = pol.staged_min;
    p->stream_min = pol.stream_min;
    return GKR_OK;
}

cudaError_t launch_insert(int32_t record, const gkr::InsertParams& p, cudaStream_t stream) {
    switch (record) {
        case 528: return gkr::launch_insert_v41(p, stream);
        case 584: return gkr::launch_insert_v4(p, stream);
        case 272: return gkr::launch_insert_mxfp4(p, stream);
        case 512: return gkr::launch_insert_fp8(p, stream);
        default: return gkr::launch_insert_bf16(p, stream);
    }
}

cudaError_t launch_gather(int32_t record, const gkr::GatherParams& p, cudaStream_t stream) {
    switch (record) {
        case 528: return gkr::launch_gather_v41(p, stream);
        case 584: return gkr::launch_gather_v4(p, stream);
        case 272: return gkr::launch_gather_mxfp4(p, stream);
        case 512: return gkr::launch_gather_fp8(p, stream);
        default: return gkr::launch_gather_bf16(p, stream);
    }
}

}  // namespace

extern "C" {

GKR_API gkr_status gkr_kv_insert(const void* kv, int64_t num_tokens, void* k_cache,
                                 const gkr_cache_desc* cache, const int64_t* slot_mapping,
                                 const int64_t* positions, const float* cos_sin_cache,
                                 int64_t max_pos, const float* fp8_scale, int32_t* err_flag,
                                 const gkr_launch_opts* opts, cudaStream_t stream) {
    gkr::InsertParams p;
    const gkr_status st = prepare_insert(kv, num_tokens, k_cache, cache, slot_mapping,
                                         positions, cos_sin_cache, max_pos, fp8_scale, err_flag,
                                         opts, &p);
    if (st != GKR_OK || p.num_tokens == 0) return st;
    return cuda_status(launch_insert(cache->record, p, stream));
}

GKR_API gkr_status gkr_rope_quant_insert(const void* kv, int64_t num_tokens, void* k_cache,
                                         const gkr_cache_desc* cache,
                                         const int64_t* slot_mapping, const int64_t* positions,
                                         const float* cos_sin_cache, int64_t max_pos,
                                         int32_t compress_ratio, int32_t sanitize_nans,
                                         int32_t* err_flag, const gkr_launch_opts* opts,
                                         cudaStream_t stream) {
    if (compress_ratio < 1 || (sanitize_nans != 0 && sanitize_nans != 1)) return GKR_EINVAL;
    if (cache != nullptr && !compressed(cache->record)) return GKR_EUNSUPPORTED_RECORD;
    gkr::InsertParams p;
    const gkr_status st = prepare_insert(kv, num_tokens, k_cache, cache, slot_mapping,
                                         positions, cos_sin_cache, max_pos, nullptr, err_flag,
                                         opts, &p);
    if (st != GKR_OK || p.num_tokens == 0) return st;
    p.ratio = compress_ratio;
    const bool san = sanitize_nans != 0;
    return cuda_status(cache->record == 528 ? gkr::launch_rope_quant_insert_v41(p, san, stream)
                                            : gkr::launch_rope_quant_insert_v4(p, san, stream));
}

GKR_API gkr_status gkr_kv_gather(const void* k_cache, const gkr_cache_desc* cache,
                                 const int32_t* indices, int64_t num_indices, void* out,
                                 const float* fp8_scale, int32_t* err_flag,
                                 const gkr_launch_opts* opts, cudaStream_t stream) {
    RecordRows rows;
    gkr_status st = check_cache(cache, &rows);
    if (st != GKR_OK) return st;
    Policy pol;
    st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (num_indices < 0) return GKR_EINVAL;
    if (num_indices == 0) return GKR_OK;
    if (!k_cache || !indices || !out) return GKR_EINVAL;
    const bool fp8 = cache->record == 512;  // fp8_scale is read for fp8 rows only
    if (fp8 && !fp8_scale) return GKR_EINVAL;
    if (!aligned(k_cache, 16) || !aligned(out, 16) || !aligned(indices, 4) ||
        !aligned(err_flag, 4) || (fp8 && !aligned(fp8_scale, 4)))
        return GKR_EALIGN;

    gkr::GatherParams p;
    p.cache = static_cast<const uint8_t*>(k_cache);
    p.page_stride = cache->page_stride;
    p.block_size = cache->block_size;
    p.num_slots = static_cast<int32_t>(cache->num_pages * cache->block_size);
    p.indices = indices;
    p.num_indices = num_indices;
    p.out = out;
    p.fp8_scale = cache->record == 512 ? fp8_scale : nullptr;
    p.err = err_flag;
    p.early_metadata = pol.early_metadata;
    p.pdl = pol.pdl;
    return cuda_status(launch_gather(cache->record, p, stream));
}

GKR_API gkr_status gkr_qnorm_rope_kv_insert(const void* q_in, int32_t num_heads,
                                            int32_t num_heads_padded, void* q_out,
                                            const float* q_scale, float eps,
                                            int32_t apply_q_norm, const void* kv,
                                            int64_t num_tokens, void* k_cache,
                                            const gkr_cache_desc* cache,
                                            const int64_t* slot_mapping,
                                            const int64_t* positions,
                                            const float* cos_sin_cache, int64_t max_pos,
                                            const float* fp8_scale, int32_t* err_flag,
                                            const gkr_launch_opts* opts,
                                            cudaStream_t stream) {
    if (num_heads < 0 || num_heads_padded < num_heads || num_heads_padded > kMaxQHeads ||
        (apply_q_norm != 0 && apply_q_norm != 1) || !(eps >= 0.0f && eps <= 3.40282347e38f))
        return GKR_EINVAL;
    gkr::InsertParams p;
    const gkr_status st = prepare_insert(kv, num_tokens, k_cache, cache, slot_mapping,
                                         positions, cos_sin_cache, max_pos, fp8_scale, err_flag,
                                         opts, &p);
    if (st != GKR_OK || p.num_tokens == 0) return st;
    if (num_heads_padded == 0) return cuda_status(launch_insert(cache->record, p, stream));
    if ((num_heads > 0 && q_in == nullptr) || q_out == nullptr) return GKR_EINVAL;
    if ((num_heads > 0 && !aligned(q_in, 16)) || !aligned(q_out, 16) ||
        (q_scale != nullptr && !aligned(q_scale, 4)))
        return GKR_EALIGN;
    if (q_scale != nullptr && num_heads > 0) {   // e4m3 rows of 512 B must not overlap q_in
        const uintptr_t in0 = reinterpret_cast<uintptr_t>(q_in);
        const uintptr_t out0 = reinterpret_cast<uintptr_t>(q_out);
        const uintptr_t in1 = in0 + static_cast<uintptr_t>(p.num_tokens) * num_heads * 1024;
        const uintptr_t out1 = out0 + static_cast<uintptr_t>(p.num_tokens) * num_heads_padded * 512;
        if (out0 < in1 && in0 < out1) return GKR_EINVAL;
    }
    gkr::QSideParams qp;
    qp.q_in = q_in;
    qp.q_out = q_out;
    qp.q_scale = q_scale;
    qp.num_heads = num_heads;
    qp.num_heads_padded = num_heads_padded;
    qp.eps = eps;
    qp.apply_norm = apply_q_norm;
    return cuda_status(gkr::launch_qnorm_rope_kv_insert(cache->record, p, qp, stream));
}

GKR_API gkr_status gkr_sparse_logits(const void* q, int32_t num_heads, const void* k_cache,
                                     const gkr_cache_desc* cache, const int32_t* indices,
                                     int64_t num_queries, int64_t topk, float sm_scale,
                                     const float* fp8_scale, float* out, int32_t* err_flag,
                                     const gkr_launch_opts* opts, cudaStream_t stream) {
    RecordRows rows;
    gkr_status st = check_cache(cache, &rows);
    if (st != GKR_OK) return st;
    if (cache->record == 272) return GKR_EUNSUPPORTED_RECORD;   // read by gkr_sparse_attention
    Policy pol;
    st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (num_queries < 0 || topk < 0 || topk % 4 != 0 || topk > INT64_C(0x7FFFFFFF) ||
        num_heads < 1 || num_heads > gkr::logits_max_heads() ||
        !(sm_scale >= -3.40282347e38f && sm_scale <= 3.40282347e38f))
        return GKR_EINVAL;
    if (num_queries == 0 || topk == 0) return GKR_OK;
    if (!q || !k_cache || !indices || !out) return GKR_EINVAL;
    const bool fp8 = cache->record == 512;
    if (fp8 && !fp8_scale) return GKR_EINVAL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(out, 16) || !aligned(indices, 4) ||
        !aligned(err_flag, 4) || (fp8 && !aligned(fp8_scale, 4)))
        return GKR_EALIGN;
    gkr::LogitsParams p;
    p.q = q;
    p.num_heads = num_heads;
    p.cache = static_cast<const uint8_t*>(k_cache);
    p.page_stride = cache->page_stride;
    p.block_size = cache->block_size;
    p.num_slots = static_cast<int32_t>(cache->num_pages * cache->block_size);
    p.indices = indices;
    p.num_queries = num_queries;
    p.topk = topk;
    const int64_t chunk = gkr::logits_chunk_keys(cache->record);
    p.chunks = (topk + chunk - 1) / chunk;
    if (num_queries > INT64_C(0x7FFFFFFF) / p.chunks) return GKR_EINVAL;   // grid < 2^31
    p.sm_scale = sm_scale;
    p.fp8_scale = fp8 ? fp8_scale : nullptr;
    p.out = out;
    p.err = err_flag;
    p.pdl = pol.pdl;
    return cuda_status(gkr::launch_sparse_logits(cache->record, p, stream));
}

GKR_API gkr_status gkr_sparse_attention_workspace(int32_t num_heads, int64_t num_queries,
                                                  int64_t topk, int64_t* bytes) {
    if (bytes == nullptr || num_heads < 1 || num_heads > gkr::kAttentionMaxHeads ||
        num_queries < 0 || num_queries > kMaxRows || topk < 0 || topk > kMaxRows)
        return GKR_EINVAL;
    *bytes = 0;
    if (num_queries == 0) return GKR_OK;
    return cuda_status(gkr::attention_workspace(num_heads, num_queries, topk, bytes));
}

GKR_API gkr_status gkr_sparse_attention(const void* q, int32_t num_heads, const void* k_cache,
                                        const gkr_cache_desc* cache, const int32_t* indices,
                                        int64_t index_stride, int64_t num_queries, int64_t topk,
                                        float sm_scale, void* out, float* lse, float* weights,
                                        int64_t weight_stride, void* workspace,
                                        int64_t workspace_bytes, int32_t* err_flag,
                                        const gkr_launch_opts* opts, cudaStream_t stream) {
    RecordRows rows;
    gkr_status st = check_cache(cache, &rows);
    if (st != GKR_OK) return st;
    if (cache->record != 272) return GKR_EUNSUPPORTED_RECORD;
    // rows of 256 bytes are counted in 32 bits
    if ((cache->page_stride >> 8) > INT64_C(0x7FFFFFFF) / cache->num_pages)
        return GKR_EBAD_PAGE_GEOMETRY;
    Policy pol;
    st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (num_queries < 0 || num_queries > kMaxRows || topk < 0 || topk > kMaxRows ||
        num_heads < 1 || num_heads > gkr::kAttentionMaxHeads || index_stride < topk ||
        (weights != nullptr && weight_stride < topk) ||
        !(sm_scale >= -3.40282347e38f && sm_scale <= 3.40282347e38f))
        return GKR_EINVAL;
    // runs of chunks (64 entries) are counted in 32 bits
    if (num_queries * ((topk + 63) / 64) > INT64_C(0x7FFFFFFF)) return GKR_EINVAL;
    if (num_queries == 0) return GKR_OK;
    if (!q || !k_cache || !out || !lse || (topk > 0 && !indices)) return GKR_EINVAL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(out, 16) || !aligned(indices, 4) ||
        !aligned(lse, 4) || !aligned(weights, 4) || !aligned(err_flag, 4))
        return GKR_EALIGN;
    int64_t need = 0;
    const cudaError_t e = gkr::attention_workspace(num_heads, num_queries, topk, &need);
    if (e != cudaSuccess) return cuda_status(e);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GKR_EINVAL;
    if (need > 0 && !aligned(workspace, 16)) return GKR_EALIGN;
    gkr::AttentionParams p;
    p.q = q;
    p.num_heads = num_heads;
    p.cache = static_cast<const uint8_t*>(k_cache);
    p.page_stride = cache->page_stride;
    p.block_size = cache->block_size;
    p.num_slots = static_cast<int32_t>(cache->num_pages * cache->block_size);
    p.indices = indices;
    p.index_stride = index_stride;
    p.num_queries = num_queries;
    p.topk = topk;
    p.sm_scale = sm_scale;
    p.out = out;
    p.lse = lse;
    p.weights = weights;
    p.weight_stride = weight_stride;
    p.workspace = workspace;
    p.err = err_flag;
    p.pdl = pol.pdl;
    return cuda_status(gkr::launch_sparse_attention(p, stream));
}

GKR_API gkr_status gkr_kv_evict(const int32_t* indices, int64_t index_stride,
                                const float* weights, int64_t weight_stride, int64_t num_rows,
                                int64_t length, int64_t keep, int64_t recent, int32_t* kept,
                                float* kept_weights, int64_t* evicted,
                                const gkr_launch_opts* opts, cudaStream_t stream) {
    Policy pol;
    const gkr_status st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (num_rows < 0 || num_rows > kMaxRows || length < 0 || length > kMaxList || keep < 0 ||
        keep > length || recent < 0 || recent > keep || index_stride < length ||
        weight_stride < length)
        return GKR_EINVAL;
    if (num_rows == 0 || length == 0) return GKR_OK;
    if (!indices || !weights || (keep > 0 && (!kept || !kept_weights)) ||
        (keep < length && !evicted))
        return GKR_EINVAL;
    if (!aligned(indices, 4) || !aligned(weights, 4) || !aligned(kept, 4) ||
        !aligned(kept_weights, 4) || !aligned(evicted, 8))
        return GKR_EALIGN;
    gkr::EvictParams p;
    p.indices = indices;
    p.index_stride = index_stride;
    p.weights = weights;
    p.weight_stride = weight_stride;
    p.rows = num_rows;
    p.length = static_cast<int32_t>(length);
    p.keep = static_cast<int32_t>(keep);
    p.recent = static_cast<int32_t>(recent);
    p.kept = kept;
    p.kept_weights = kept_weights;
    p.evicted = evicted;
    p.pdl = pol.pdl;
    return cuda_status(gkr::launch_evict(p, stream));
}

GKR_API gkr_status gkr_kv_allocate(const int32_t* past, const int32_t* added,
                                   int32_t num_requests, int32_t* block_table,
                                   int64_t table_stride, int32_t table_width,
                                   const int32_t* free_pages, int64_t num_free,
                                   int32_t block_size, int64_t num_tokens, int64_t* slot_mapping,
                                   int64_t* positions, int32_t* starts, int32_t* taken,
                                   int32_t* err_flag, const gkr_launch_opts* opts,
                                   cudaStream_t stream) {
    Policy pol;
    const gkr_status st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (num_requests < 0 || num_requests > gkr::kPlanMaxRequests || table_width < 0 ||
        table_stride < table_width || num_free < 0 || num_free > kMaxIndex || block_size < 1 ||
        num_tokens < 0 || num_tokens > kMaxIndex)
        return GKR_EINVAL;
    if ((num_requests > 0 && (!past || !added || (table_width > 0 && !block_table))) ||
        (num_free > 0 && !free_pages) || (num_tokens > 0 && (!slot_mapping || !positions)) ||
        !starts || !taken)
        return GKR_EINVAL;
    if (!aligned(past, 4) || !aligned(added, 4) || !aligned(block_table, 4) ||
        !aligned(free_pages, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 8) ||
        !aligned(starts, 4) || !aligned(taken, 4) || !aligned(err_flag, 4))
        return GKR_EALIGN;
    gkr::AllocateParams p;
    p.past = past;
    p.added = added;
    p.num_requests = num_requests;
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_width = table_width;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.block_size = block_size;
    p.num_tokens = num_tokens;
    p.slots = slot_mapping;
    p.positions = positions;
    p.starts = starts;
    p.taken = taken;
    p.err = err_flag;
    p.pdl = pol.pdl;
    return cuda_status(gkr::launch_allocate(p, stream));
}

GKR_API gkr_status gkr_kv_slots(const int32_t* block_table, int64_t table_stride,
                                int32_t table_width, const int32_t* lengths,
                                const int32_t* first, int32_t num_requests, int32_t block_size,
                                int64_t width, int32_t* indices, int32_t* starts,
                                int32_t* err_flag, const gkr_launch_opts* opts,
                                cudaStream_t stream) {
    Policy pol;
    const gkr_status st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    const bool packed_rows = starts != nullptr;
    if (num_requests < 0 || table_width < 0 || table_stride < table_width || block_size < 1 ||
        width < 0 || width > kMaxIndex || (packed_rows && num_requests > gkr::kPlanMaxRequests))
        return GKR_EINVAL;
    // blocks of a launch
    if (!packed_rows && width > 0 && num_requests > kMaxIndex / ((width + 2047) / 2048))
        return GKR_EINVAL;
    // without room for entries only the lengths are looked at, for the error bits
    if (!packed_rows && (num_requests == 0 || (width == 0 && !err_flag))) return GKR_OK;
    if ((num_requests > 0 && (!lengths || (table_width > 0 && !block_table))) ||
        (width > 0 && !indices))
        return GKR_EINVAL;
    if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(first, 4) ||
        !aligned(indices, 4) || !aligned(starts, 4) || !aligned(err_flag, 4))
        return GKR_EALIGN;
    gkr::SlotsParams p;
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_width = table_width;
    p.lengths = lengths;
    p.first = first;
    p.num_requests = num_requests;
    p.block_size = block_size;
    p.indices = indices;
    p.width = width;
    p.starts = starts;
    p.err = err_flag;
    p.pdl = pol.pdl;
    return cuda_status(gkr::launch_slots(p, stream));
}

GKR_API gkr_status gkr_prompt_attention_workspace(int32_t num_heads, int64_t num_tokens,
                                                  int64_t* bytes) {
    if (bytes == nullptr || !prompt_rows_ok(num_heads, num_tokens)) return GKR_EINVAL;
    *bytes = 0;
    if (num_tokens == 0) return GKR_OK;
    return cuda_status(gkr::prompt_workspace(num_heads, num_tokens, bytes));
}

GKR_API gkr_status gkr_prompt_attention(const void* q, int32_t num_heads, int64_t num_tokens,
                                        const void* kv, int64_t kv_stride, int64_t num_rows,
                                        const int32_t* starts, const int32_t* kv_starts,
                                        int32_t num_requests, int32_t causal, float sm_scale,
                                        void* out, float* lse, void* workspace,
                                        int64_t workspace_bytes, int32_t* err_flag,
                                        const gkr_launch_opts* opts, cudaStream_t stream) {
    Policy pol;
    const gkr_status st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (!prompt_rows_ok(num_heads, num_tokens) || num_rows < 0 || num_rows > kMaxPromptRows ||
        kv_stride < 512 || kv_stride > (INT64_C(1) << 34) || kv_stride % 8 != 0 ||
        num_rows > (INT64_C(1) << 37) / num_heads ||
        num_requests < 0 || num_requests > gkr::kPlanMaxRequests || causal < 0 || causal > 1 ||
        !finite(sm_scale))
        return GKR_EINVAL;
    if (num_tokens == 0 || num_requests == 0) return GKR_OK;
    if (!q || (num_rows > 0 && !kv) || !starts || !kv_starts || !out || !lse) return GKR_EINVAL;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(starts, 4) || !aligned(kv_starts, 4) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(err_flag, 4))
        return GKR_EALIGN;
    const int64_t out_bytes = num_tokens * num_heads * 1024;
    if (overlap(out, out_bytes, q, out_bytes) ||
        (num_rows > 0 && overlap(out, out_bytes, kv, ((num_rows - 1) * kv_stride + 512) * 2)))
        return GKR_EINVAL;
    int64_t need = 0;
    const cudaError_t e = gkr::prompt_workspace(num_heads, num_tokens, &need);
    if (e != cudaSuccess) return cuda_status(e);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GKR_EINVAL;
    if (need > 0 && !aligned(workspace, 16)) return GKR_EALIGN;
    gkr::PromptParams p;
    p.q = q;
    p.num_heads = num_heads;
    p.num_tokens = num_tokens;
    p.kv = kv;
    p.kv_stride = kv_stride;
    p.num_rows = num_rows;
    p.starts = starts;
    p.kv_starts = kv_starts;
    p.num_requests = num_requests;
    p.causal = causal;
    p.sm_scale = sm_scale;
    p.out = out;
    p.lse = lse;
    p.workspace = workspace;
    p.err = err_flag;
    p.pdl = pol.pdl;
    return cuda_status(gkr::launch_prompt_attention(p, stream));
}

GKR_API gkr_status gkr_prefix_attention_workspace(int32_t num_heads, int64_t num_queries,
                                                  int64_t prefix_length, int64_t topk,
                                                  int64_t* bytes) {
    if (bytes == nullptr || !prefix_sizes_ok(num_heads, num_queries, prefix_length, topk))
        return GKR_EINVAL;
    *bytes = 0;
    if (num_queries == 0) return GKR_OK;
    return cuda_status(gkr::prefix_workspace(num_heads, num_queries, prefix_length, topk, bytes));
}

GKR_API gkr_status gkr_prefix_attention(const void* q, int32_t num_heads, const void* k_cache,
                                        const gkr_cache_desc* cache, const int32_t* prefix,
                                        int64_t prefix_length, const int32_t* indices,
                                        int64_t index_stride, int64_t num_queries, int64_t topk,
                                        float sm_scale, void* out, float* lse, void* workspace,
                                        int64_t workspace_bytes, int32_t* err_flag,
                                        const gkr_launch_opts* opts, cudaStream_t stream) {
    RecordRows rows;
    gkr_status st = check_cache(cache, &rows);
    if (st != GKR_OK) return st;
    if (cache->record != 272) return GKR_EUNSUPPORTED_RECORD;
    // rows of 256 bytes are counted in 32 bits
    if ((cache->page_stride >> 8) > INT64_C(0x7FFFFFFF) / cache->num_pages)
        return GKR_EBAD_PAGE_GEOMETRY;
    Policy pol;
    st = resolve_policy(opts, &pol);
    if (st != GKR_OK) return st;
    if (!prefix_sizes_ok(num_heads, num_queries, prefix_length, topk) || index_stride < topk ||
        !finite(sm_scale))
        return GKR_EINVAL;
    if (num_queries == 0) return GKR_OK;
    if (!q || !k_cache || !out || !lse || (prefix_length > 0 && !prefix) || (topk > 0 && !indices))
        return GKR_EINVAL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(out, 16) || !aligned(prefix, 4) ||
        !aligned(indices, 4) || !aligned(lse, 4) || !aligned(err_flag, 4))
        return GKR_EALIGN;
    const int64_t out_bytes = num_queries * num_heads * 1024;
    if (overlap(out, out_bytes, q, out_bytes)) return GKR_EINVAL;
    int64_t need = 0;
    const cudaError_t e =
        gkr::prefix_workspace(num_heads, num_queries, prefix_length, topk, &need);
    if (e != cudaSuccess) return cuda_status(e);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GKR_EINVAL;
    if (need > 0 && !aligned(workspace, 16)) return GKR_EALIGN;
    gkr::PrefixParams p;
    p.own.q = q;
    p.own.num_heads = num_heads;
    p.own.cache = static_cast<const uint8_t*>(k_cache);
    p.own.page_stride = cache->page_stride;
    p.own.block_size = cache->block_size;
    p.own.num_slots = static_cast<int32_t>(cache->num_pages * cache->block_size);
    p.own.indices = indices;
    p.own.index_stride = index_stride;
    p.own.num_queries = num_queries;
    p.own.topk = topk;
    p.own.sm_scale = sm_scale;
    p.own.out = out;
    p.own.lse = lse;
    p.own.weights = nullptr;
    p.own.weight_stride = 0;
    p.own.workspace = workspace;
    p.own.err = err_flag;
    p.own.pdl = pol.pdl;
    p.prefix = prefix;
    p.prefix_length = prefix_length;
    return cuda_status(gkr::launch_prefix_attention(p, stream));
}

GKR_API const char* gkr_status_string(gkr_status status) {
    switch (status) {
        case GKR_OK: return "ok";
        case GKR_EINVAL: return "invalid argument";
        case GKR_EUNSUPPORTED_RECORD:
            return "unsupported record width (expected 528 or 584, 512 / 1024 for the fp8 and "
                   "bf16 caches, or 272 for MXFP4; the compressed insert writes 528 / 584 "
                   "only, the sparse logits read all but 272, the sparse attention 272 only)";
        case GKR_EBAD_PAGE_GEOMETRY:
            return "bad page geometry (page_stride below block_size * record or not a "
                   "multiple of the record's page alignment: 576 for 584, else 512)";
        case GKR_EALIGN: return "misaligned pointer";
        case GKR_ECUDA: return "CUDA launch error";
    }
    return "unknown status";
}

GKR_API int32_t gkr_last_cuda_error(void) { return g_last_cuda_error; }

GKR_API int32_t gkr_version(void) { return 30200; }

}  // extern "C"
