// What the attention kernels share: the softmax's constants and exponentials, 16-byte accesses
// to shared memory, barriers of a group of warps, and the mark of results that were left out.
#pragma once

#include "tensor.cuh"

namespace gkr {

namespace {

constexpr int32_t kErrIndex = 4;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;


// A new maximum replaces the running one only when it is this much larger (in powers of two), for
// any of the 32 heads of a warp: rescaling the accumulator takes longer than a chunk's softmax
// (1400 cycles), and at 8, with the logits of heavy-tailed latents, every second chunk had some
// head that rose.  The reference does not touch the precision of floating-point terms, only
// their range: probabilities stay below 2^(kLag + kLift) = 2^48, so an output cannot overflow while the
// number of rows times the largest value is below 2^80 (2^24 records, the most of a list: 2^55 each).
constexpr float kLag = 32.0f;
// Where the reference moves up by 2^-by, what is in the accumulator is multiplied by 2^(by / 2) twice: its terms may
// lie 2^(kLag + kLift) above the old reference and still count where 2^by is below what fp32 holds (one
// factor lost what had weights of up to 2^-117).  The sums of the probabilities end far above that.
// Probabilities are taken as exp2(s - m + kLift): bf16 ends at 2^-133, and without the lift terms
// that the output still shows (it ends there too) would be rounded away before they are
// multiplied by a record's values and summed.
constexpr float kLift = 16.0f;

// The lse of a query, or of a piece, whose results are not written because a wait gave up
// (kErrTimeout): a NaN that no instruction produces, so that the kernels that follow can tell it
// from the NaN of a record.
constexpr uint32_t kUnwritten = 0x7FC0B0B0u;
__device__ __forceinline__ bool is_unwritten(float lse) { return __float_as_uint(lse) == kUnwritten; }

// 2^x within 2^-22; results below 2^-126 kept (factors that rescale what may be large) ...
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// ... or, in one instruction, flushed to zero (a probability: kLift puts those below 2^-142).
__device__ __forceinline__ float exp2_flush(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16_at(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// A stage of a ring and the parity of its current round.
template <int N>
struct Ring {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ void skip(int n) {
        const uint32_t at = static_cast<uint32_t>(s) + static_cast<uint32_t>(n);
        parity ^= at / N & 1u;
        s = static_cast<int>(at % N);
    }
};

// A barrier of the first `threads` threads that come to it.
__device__ __forceinline__ void group_sync(int bar, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
}

// The same, and whether any of the threads says so.
__device__ __forceinline__ bool group_any(int bar, int threads, bool mine) {
    uint32_t any;
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n barrier.red.or.pred p, %2, %3, p;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(any)
                 : "r"(mine ? 1u : 0u), "r"(bar), "r"(threads) : "memory");
    return any != 0u;
}

// Eight fp32 values as bf16, and scaled.
__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                      pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack8(const float* v, float f) {
    return make_uint4(pack_bf16x2_rn(__fmul_rn(v[0], f), __fmul_rn(v[1], f)),
                      pack_bf16x2_rn(__fmul_rn(v[2], f), __fmul_rn(v[3], f)),
                      pack_bf16x2_rn(__fmul_rn(v[4], f), __fmul_rn(v[5], f)),
                      pack_bf16x2_rn(__fmul_rn(v[6], f), __fmul_rn(v[7], f)));
}

// The sum of those eight as they are after the rounding; its two halves are still to be added.
__device__ __forceinline__ uint64_t sum_rounded(uint4 w) {
    auto two = [](uint32_t x) { return f32x2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)); };
    return add_f32x2(add_f32x2(two(w.x), two(w.y)), add_f32x2(two(w.z), two(w.w)));
}

}  // namespace
}  // namespace gkr
