// Helpers shared by the embedding head's kernels.
#pragma once

#include <type_traits>

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

// A float of its bits. (Applied to an element of a vector in place, the bit cast of
// ROCm 7.2 takes element 0 whatever the index.)
__device__ __forceinline__ float as_float(uint32_t bits) { return __builtin_bit_cast(float, bits); }

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

// f(integral_constant<int, I>) for I = B .. E-1, unrolled at compile time
template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f)
{
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

// R (4 or 16) consecutive outputs n .. n + R - 1 of row t, those below N, in
// pieces of up to 16 bytes where N keeps every row aligned for them. zero:
// zeros in place of y, whatever it holds.
template <int R>
__device__ __forceinline__ void store_run(void* Y, int out, int64_t t, int n, int N, const float (&y)[R],
                                          bool zero = false)
{
    const int64_t at = t * N + n;
    if (out == kF32) {
        float* p = (float*)Y + at;
        float v[R];
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = zero ? 0.0f : y[i];
        if ((N & 3) == 0) {
#pragma unroll
            for (int i = 0; i < R / 4; ++i)
                if (n + 4 * i < N) ((f32x4*)p)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (n + i < N) p[i] = v[i];
        }
        return;
    }
    uint16_t* p = (uint16_t*)Y + at;
    uint32_t w[R / 2];
    if (out == kBF16) {
#pragma unroll
        for (int i = 0; i < R / 2; ++i) w[i] = half_pair<kBF16>(y[2 * i], y[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < R / 2; ++i) w[i] = half_pair<kF16>(y[2 * i], y[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < R / 2; ++i) w[i] = zero ? 0 : w[i];
    if (R == 16 && (N & 7) == 0) {
#pragma unroll
        for (int i = 0; i < R / 8; ++i)
            if (n + 8 * i < N) ((u32x4*)p)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    } else if ((N & 3) == 0) {
#pragma unroll
        for (int i = 0; i < R / 4; ++i)
            if (n + 4 * i < N) ((u32x2*)p)[i] = u32x2{w[2 * i], w[2 * i + 1]};
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (n + i < N) p[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
    }
}

// Four dma_lds16 (NT: with the non-temporal hint) from one base to four KB in a
// row of LDS; they share the wait states behind the base. Against four single
// loads, 200,000 x 2048 to 256 channels take 167.7 instead of 181.3 us and
// 8192 x 4096 x 4096 125.0 instead of 127.0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
#define MAXSIM_DMA4(HINT)                                                                                    \
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %5" HINT                       \
                 "\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %5" HINT            \
                 "\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %5" HINT            \
                 "\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %5" HINT            \
                 :                                                                                           \
                 : "s"(lds), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(base)               \
                 : "memory", "m0", "scc")
template <bool NT>
__device__ __forceinline__ void dma_lds16_x4(const void* base, const uint32_t* voff, uint32_t lds)
{
    if constexpr (NT) MAXSIM_DMA4(" nt");
    else MAXSIM_DMA4("");
}
#undef MAXSIM_DMA4
#pragma clang diagnostic pop

// position of 16-byte chunk c of a row of KB bytes, against bank conflicts
template <int KB>
__device__ __forceinline__ int place(int row, int c)
{
    if constexpr (KB >= 128) return swz_chunk<KB>(row, c);
    else return c ^ ((row >> 2) & 3);  // 64-byte rows: four share a 256-byte bank line
}

// Which channel of its 32 an MFMA row stands for. A lane's 16 results are rows
// 8 b + 4 h + e of its half h; with this order they are 16 consecutive channels,
// 16 h + 4 b + e, and are stored as one run.
__device__ __forceinline__ int channel_of(int row)
{
    return (row & ~31) | (row & 4) << 2 | (row & 24) >> 1 | (row & 3);
}

}  // namespace maxsim
