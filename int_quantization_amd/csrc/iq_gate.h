// Device pieces shared by the gated block's kernels: vector types, BF16
// packing, the activations and their slopes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "iq_ffn_launch.h"

namespace iqk {
namespace gate {

typedef float f4v __attribute__((ext_vector_type(4)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

// FP32 to BF16, to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const bf2v v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ f4v mfma(bf8v a, bf8v b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Workgroup barrier that orders LDS only: outstanding global accesses stay
// in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits until at most N loads and copies of the wave are outstanding.
template <int N> __device__ __forceinline__ void wait_for_all_but() {
    static_assert(N < 64, "six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    asm volatile("" ::: "memory");
}

// 1 / (1 + e^-v), also for both infinities.  The exponential is the hardware's
// power of two: its argument, v times log2 e, is rounded once, which costs a
// relative |v| 2^-24, as much as rounding v itself to FP32 did.
__device__ __forceinline__ float logistic(float v) { return 1.f / (1.f + __expf(-v)); }

constexpr float kTanhC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// act(g).  GELU's tanh form uses (1 + tanh z) / 2 = 1 / (1 + e^-2z), and the
// exact one (1 + erf z) / 2 = erfc(-z) / 2: from g = -3 on 1 + erf has lost
// digits, at -6 all.
template <int ACT> __device__ __forceinline__ float act(float g) {
    if constexpr (ACT == A_SILU) return g * logistic(g);
    if constexpr (ACT == A_GELU) return 0.5f * g * erfcf(g * -0.7071067811865476f);
    return g * logistic(2.f * kTanhC * (g + kTanhA * g * g * g));
}

// act(g) and act'(g).
template <int ACT> __device__ __forceinline__ void act_slope(float g, float& a, float& da) {
    if constexpr (ACT == A_SILU) {
        const float p = logistic(g);
        a = g * p;
        da = p + a * (1.f - p);
    } else if constexpr (ACT == A_GELU) {
        const float p = 0.5f * erfcf(g * -0.7071067811865476f);
        a = g * p;
        da = p + g * __expf(-0.5f * g * g) * 0.3989422804014327f;
    } else {
        const float p = logistic(2.f * kTanhC * (g + kTanhA * g * g * g));
        a = g * p;
        // beyond 100 p is 0 or 1 and the product 0, also where g g would be infinite
        da = p + a * (1.f - p) * 2.f * kTanhC * (1.f + 3.f * kTanhA * fminf(g * g, 1e4f));
    }
}

}  // namespace gate
}  // namespace iqk
