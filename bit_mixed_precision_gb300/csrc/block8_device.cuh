// Device helpers of the 8-bit block cache (block8_*): the quantiser, the
// queries' limits, exact conversions of 8-bit codes to fp16 pairs.
#pragma once

#include "kvq_common.cuh"

namespace kvq {
namespace b8 {

constexpr float kSmallestScale = 5.421010862427522e-20f;    // 2^-64

// Largest code magnitude and its rounded reciprocal (the quantiser multiplies by it).
template <int CODE> struct Code;
template <> struct Code<KVQ_CODE_E4M3> {
    static constexpr float kInvMax = 1.0f / 448.0f;
};
template <> struct Code<KVQ_CODE_INT8> {
    static constexpr float kInvMax = 1.0f / 127.0f;
};
constexpr float kInv127 = 1.0f / 127.0f;

__device__ __forceinline__ float scale_of(float amax, float inv_max) {
    return fmaxf(__fmul_rn(amax, inv_max), kSmallestScale);
}

// Two codes of RN(x * inv), x0's in the low byte.
template <int CODE>
__device__ __forceinline__ uint32_t code_pair(float x0, float x1, float inv) {
    const float a = __fmul_rn(x0, inv), b = __fmul_rn(x1, inv);
    if constexpr (CODE == KVQ_CODE_E4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    } else {
        const int ia = min(127, max(-127, __float2int_rn(a))), ib = min(127, max(-127, __float2int_rn(b)));
        return (uint32_t)(ia & 255) | ((uint32_t)(ib & 255) << 8);
    }
}

// Rows of the call that sequence b has; a bad entry is clamped and reported.
__device__ __forceinline__ int new_rows(const int32_t* n_new, int b, int n, uint32_t* status) {
    if (n_new == nullptr) return n;
    const int m = n_new[b];
    if (m >= 0 && m <= n) return m;
    atomicOr(status, kDevCheck);
    return m < 0 ? 0 : n;
}

// Tokens of a unit with count tokens that query t of m sees.
__device__ __forceinline__ int query_limit(int count, int m, int t) { return t < m ? max(0, count - m + t + 1) : 0; }

// Key of a score for top-k: NaN above everything, -0 equal to +0.
__device__ __forceinline__ uint32_t rank_key(float f) {
    if (isnan(f)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace b8
}  // namespace kvq
