// Attention of packed prompts over packed latent rows, and decode attention behind a shared
// prefix.  First form: a warp for each query head, one row at a time.
#include <cmath>

#include "decode.cuh"
#include "device.cuh"
#include "launch.h"

namespace gkr {

namespace {

constexpr int32_t kErrIndex = 4;
constexpr int kRowThreads = 256;

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// A query head's softmax and sum over the rows it is given one after another; lane L has
// dims [8L, 8L + 8) and [256 + 8L, 256 + 8L + 8).
struct RowState {
    float q[16], acc[16], m, l;
    __device__ void init(const uint8_t* qrow, int lane, float sm_scale) {
        unpack_bf16x8(*reinterpret_cast<const uint4*>(qrow + 16 * lane), q);
        unpack_bf16x8(*reinterpret_cast<const uint4*>(qrow + 512 + 16 * lane), q + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
        m = -INFINITY;
        l = 0.0f;
        scale = sm_scale;
    }
    __device__ void add(const uint4 a, const uint4 b) {
        float k[16], s = 0.0f;
        unpack_bf16x8(a, k);
        unpack_bf16x8(b, k + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) s = __fmaf_rn(q[i], k[i], s);
        s = __fmul_rn(warp_add(s), scale);
        const float top = fmaxf(m, s);
        const float ref = top == -INFINITY ? 0.0f : top;
        const float fix = expf(__fsub_rn(m, ref)), p = expf(__fsub_rn(s, ref));
        m = top;
        l = __fmaf_rn(l, fix, p);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = __fmaf_rn(acc[i], fix, __fmul_rn(p, k[i]));
    }
    __device__ void write(uint8_t* out, float* lse, int lane) {
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = pack_bf16x2_rn(__fmul_rn(acc[2 * i], inv), __fmul_rn(acc[2 * i + 1], inv));
        st16(out + 16 * lane, make_uint4(w[0], w[1], w[2], w[3]));
        st16(out + 512 + 16 * lane, make_uint4(w[4], w[5], w[6], w[7]));
        if (lane == 0) *lse = l == 0.0f ? -INFINITY : __fadd_rn(m, logf(l));
    }
    float scale;
};

__global__ void __launch_bounds__(kRowThreads) prompt_kernel(const PromptParams p) {
    const int lane = threadIdx.x & 31;
    pdl_wait_previous();
    pdl_release_next();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = row / p.num_heads;
    if (t >= p.num_tokens) return;
    for (int b = 0; b < p.num_requests; ++b) {
        const int64_t q0 = min(max(static_cast<int64_t>(p.starts[b]), INT64_C(0)), p.num_tokens);
        const int64_t q1 = min(max(static_cast<int64_t>(p.starts[b + 1]), q0), p.num_tokens);
        const int64_t k0 = min(max(static_cast<int64_t>(p.kv_starts[b]), INT64_C(0)), p.num_rows);
        const int64_t k1 = min(max(static_cast<int64_t>(p.kv_starts[b + 1]), k0), p.num_rows);
        if (lane == 0 && row == 0 &&
            (q0 != p.starts[b] || q1 != p.starts[b + 1] || k0 != p.kv_starts[b] || k1 != p.kv_starts[b + 1]))
            report(p.err, kErrIndex);
        if (t < q0 || t >= q1) continue;
        const int64_t see = p.causal ? max((k1 - k0) - (q1 - q0) + (t - q0) + 1, INT64_C(0)) : k1 - k0;
        RowState s;
        s.init(static_cast<const uint8_t*>(p.q) + row * 1024, lane, p.sm_scale);
        const uint8_t* k = static_cast<const uint8_t*>(p.kv) + k0 * p.kv_stride * 2 + 16 * lane;
        for (int64_t i = 0; i < see; ++i, k += p.kv_stride * 2)
            s.add(*reinterpret_cast<const uint4*>(k), *reinterpret_cast<const uint4*>(k + 512));
        s.write(static_cast<uint8_t*>(p.out) + row * 1024, p.lse + row, lane);
    }
}

__global__ void __launch_bounds__(kRowThreads) prefix_kernel(const PrefixParams p) {
    const int lane = threadIdx.x & 31;
    pdl_wait_previous();
    pdl_release_next();
    const AttentionParams& a = p.own;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t i = row / a.num_heads;
    if (i >= a.num_queries) return;
    RowState s;
    s.init(static_cast<const uint8_t*>(a.q) + row * 1024, lane, a.sm_scale);
    bool bad = false;
    const auto list = [&](const int32_t* idx, int64_t n) {
        for (int64_t k = 0; k < n; ++k) {
            const int32_t slot = idx[k];
            if (slot < 0 || slot >= a.num_slots) {
                bad |= slot != -1;
                continue;
            }
            uint32_t page, at;
            page_row(static_cast<uint32_t>(slot), static_cast<uint32_t>(a.block_size), page, at);
            const uint8_t* const base = a.cache + page * a.page_stride;
            const uint8_t* const data = base + at * 256u + 4 * lane;
            const uint8_t* const scale = base + static_cast<int64_t>(a.block_size) * 256 + at * 16u + (lane >> 2);
            s.add(dequant8_e2m1(*reinterpret_cast<const uint32_t*>(data), e2m1_factor(scale[0])),
                  dequant8_e2m1(*reinterpret_cast<const uint32_t*>(data + 128), e2m1_factor(scale[8])));
        }
    };
    list(p.prefix, p.prefix_length);
    list(a.indices + i * a.index_stride, a.topk);
    if (bad && lane == 0) report(a.err, kErrIndex);
    s.write(static_cast<uint8_t*>(a.out) + row * 1024, a.lse + row, lane);
}

int64_t row_blocks(int64_t rows) { return (rows + kRowThreads / 32 - 1) / (kRowThreads / 32); }

}  // namespace

cudaError_t prompt_workspace(int32_t, int64_t, int64_t* bytes) {
    *bytes = 0;
    return cudaSuccess;
}

cudaError_t prefix_workspace(int32_t, int64_t, int64_t, int64_t, int64_t* bytes) {
    *bytes = 0;
    return cudaSuccess;
}

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t stream) {
    return launch_kernel(prompt_kernel, row_blocks(p.num_tokens * p.num_heads), kRowThreads, 0, stream, p.pdl, p);
}

cudaError_t launch_prefix_attention(const PrefixParams& p, cudaStream_t stream) {
    return launch_kernel(prefix_kernel, row_blocks(p.own.num_queries * p.own.num_heads), kRowThreads, 0, stream,
                         p.own.pdl, p);
}

}  // namespace gkr
