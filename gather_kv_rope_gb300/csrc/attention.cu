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
// One pass over the records with a running maximum and sum: a block takes one query and eight
// heads, one head a warp; tiles of 32 records are dequantised once into shared memory for the
// eight.
#include <cmath>

#include "device.cuh"
#include "launch.h"

namespace gkr {

namespace {

constexpr int kHeadsPerBlock = 8;
constexpr int kTile = 32;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int32_t kErrIndex = 4;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, d));
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
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

__global__ void __launch_bounds__(kHeadsPerBlock * 32) attention_kernel(const AttentionParams p,
                                                                        const int groups) {
    __shared__ __align__(16) uint8_t rows[kTile * 1024];
    __shared__ uint32_t valid;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t qi = blockIdx.x / groups;
    const int h = static_cast<int>(blockIdx.x % groups) * kHeadsPerBlock + warp;
    pdl_wait_previous();
    pdl_release_next();
    const bool mine = h < p.num_heads;
    float x[16], acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = x[i] = 0.0f;
    if (mine) load_head(p, qi, h, lane, x);
    const float scale = __fmul_rn(p.sm_scale, kLog2e);   // logits in powers of two
    float m = -INFINITY, l = 0.0f;
    for (int64_t k0 = 0; k0 < p.topk; k0 += kTile) {
        const uint32_t live = load_tile(p, qi, k0, rows, &valid, warp, lane);
        if (live == 0u) continue;
        float s = -INFINITY;   // lane k: entry k0 + k
        for (int k = 0; k < kTile; ++k) {
            const float d = dot(x, rows + k * 1024, lane);
            if (lane == k && ((live >> k) & 1u) != 0u) s = __fmul_rn(d, scale);
        }
        const float top = fmaxf(m, warp_max(s));
        const float ref = top == -INFINITY ? 0.0f : top;
        const float fix = exp2_approx(__fsub_rn(m, ref));
        const float e = exp2_approx(__fsub_rn(s, ref));
        l = __fmaf_rn(l, fix, warp_sum(e));
        m = top;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = __fmul_rn(acc[i], fix);
        for (int k = 0; k < kTile; ++k) {
            const float w = __shfl_sync(kFull, e, k);
            float v[16];
            unpack_bf16x8(lds16(rows + k * 1024 + 16 * lane), v);
            unpack_bf16x8(lds16(rows + k * 1024 + 512 + 16 * lane), v + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = __fmaf_rn(w, v[i], acc[i]);
        }
    }
    if (!mine) return;
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
    uint8_t* const out = static_cast<uint8_t*>(p.out) + (qi * p.num_heads + h) * 1024;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = l == 0.0f ? 0.0f : __fmul_rn(acc[i], inv);
    st16(out + 16 * lane, make_uint4(pack_bf16x2_rn(acc[0], acc[1]), pack_bf16x2_rn(acc[2], acc[3]),
                                     pack_bf16x2_rn(acc[4], acc[5]), pack_bf16x2_rn(acc[6], acc[7])));
    st16(out + 512 + 16 * lane,
         make_uint4(pack_bf16x2_rn(acc[8], acc[9]), pack_bf16x2_rn(acc[10], acc[11]),
                    pack_bf16x2_rn(acc[12], acc[13]), pack_bf16x2_rn(acc[14], acc[15])));
    if (lane == 0) p.lse[qi * p.num_heads + h] = l == 0.0f ? -INFINITY : __fmul_rn(m + log2f(l), kLn2);
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

}  // namespace

cudaError_t attention_workspace(int32_t, int64_t, int64_t, int64_t* bytes) {
    *bytes = 0;
    return cudaSuccess;
}

cudaError_t launch_sparse_attention(const AttentionParams& p, cudaStream_t stream) {
    const int groups = (p.num_heads + kHeadsPerBlock - 1) / kHeadsPerBlock;
    cudaError_t e = launch_kernel(attention_kernel, p.num_queries * groups, kHeadsPerBlock * 32, 0,
                                  stream, p.pdl, p, groups);
    if (e != cudaSuccess || p.weights == nullptr || p.topk == 0) return e;
    const int64_t tiles = (p.topk + kTile - 1) / kTile;
    return launch_kernel(weight_kernel, p.num_queries * tiles, kHeadsPerBlock * 32, 0, stream,
                         p.pdl, p, tiles);
}

}  // namespace gkr
