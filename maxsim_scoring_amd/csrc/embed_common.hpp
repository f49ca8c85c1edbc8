// Helpers shared by the embedding head's kernels.
#pragma once

#include "common.hpp"

namespace maxsim {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Rows whose largest magnitude is below this count as zeros: the reciprocals of
// larger ones, and of their sums of squares over it, are ordinary floats.
constexpr float kTiny = 0x1p-110f;

// 1 / sqrt(x): the hardware's, off by up to 2^-23 relative, and one Newton step.
__device__ __forceinline__ float rsqrt_f(float x)
{
    const float r = __builtin_amdgcn_rsqf(x);
    return __builtin_fmaf(0.5f * r, __builtin_fmaf(-x * r, r, 1.0f), r);
}

// The bits of v rounded to the 16-bit type `out` (kBF16 or kF16).
__device__ __forceinline__ uint32_t half_bits(int out, float v)
{
    return out == kBF16 ? (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v)
                        : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
}

// Two values rounded to the 16-bit type `out`, the first in the low half.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
template <int OUT>
__device__ __forceinline__ uint32_t half_pair(float a, float b)
{
    if constexpr (OUT == kBF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}

}  // namespace maxsim
