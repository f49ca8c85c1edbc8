// Rows of floats to microscaled 4-bit codes, and back, for gfx950.
//
//   e = floor(log2 max|v|) - 2 of each block of 32,  code = E2M1 nearest to v / 2^e
//
// Both directions are bound by memory: a lane takes 8 consecutive values (16
// bytes of a 16-bit type), a quad of lanes a block, whose largest magnitude is two
// DPP steps; the codes of 8 values are one word, made by the hardware's conversion
// (nearest, ties to even, saturating: all 7 borders between levels and the values
// next to them were compared with the definition, at exponents from -127 to 127).
// Without normalisation blocks are independent and pass once.
//
// With normalisation a row's squares are summed in float64 while the row stays in
// registers. A code is decided on the quotient x / ||x||, and one that falls on
// the wrong side of a border is a whole step off, so the float32 quotient (off by
// less than 2 units in the last place) is used only where it is further than 4
// from every border; the others are formed again in float64.
#include "mx4_common.hpp"

namespace maxsim {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 22;  // blocks x threads stays far below 2^32
constexpr int kZeroScale = 127, kNanScale = 255;

template <int E> constexpr int elem_bytes() { return E == kF32 ? 4 : 2; }

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // at any element

// 8 values c .. c + 7 of a row of d, zeros behind its end. WHOLE: d is a multiple of 8.
template <int E, bool WHOLE>
__device__ __forceinline__ void load8(const void* X, int64_t row, int d, int c, float (&x)[8])
{
    const char* p = (const char*)X + (row * d + c) * elem_bytes<E>();
    if (WHOLE ? c >= d : c + 8 > d) {  // (the last block may reach past the row)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = 0.0f;
            if (WHOLE) continue;
            if (c + i < d) {
                if constexpr (E == kF32) x[i] = ((const float*)p)[i];
                else if constexpr (E == kBF16) x[i] = __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
                else x[i] = (float)((const _Float16*)p)[i];
            }
        }
        return;
    }
    u32x4 w[E == kF32 ? 2 : 1];
#pragma unroll
    for (int j = 0; j < (E == kF32 ? 2 : 1); ++j) {
        if constexpr (WHOLE) w[j] = ((const u32x4*)p)[j];
        else w[j] = ((const u32x4_any*)p)[j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (E == kF32) {
            x[i] = as_float(w[0][i]);
            x[4 + i] = as_float(w[E == kF32 ? 1 : 0][i]);
        } else if constexpr (E == kBF16) {
            x[2 * i] = as_float(w[0][i] << 16);
            x[2 * i + 1] = as_float(w[0][i] & 0xffff0000u);
        } else {
            x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[0][i] & 0xffffu));
            x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[0][i] >> 16));
        }
    }
}

// The largest of four lanes' values, NaN where one is.
template <int CTRL>
__device__ __forceinline__ float quad_step(float v)
{
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false);
    return __builtin_elementwise_maximum(v, __builtin_bit_cast(float, o));
}
__device__ __forceinline__ float quad_max(float v) { return quad_step<0x4E>(quad_step<0xB1>(v)); }

__device__ __forceinline__ float max8(const float (&x)[8])
{
    float m = __builtin_fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __builtin_elementwise_maximum(m, __builtin_fabsf(x[i]));
    return m;
}

__device__ __forceinline__ int clamp_exp(int e) { return e < -127 ? -127 : e > 127 ? 127 : e; }

// 2^e, e in [-127, 127]
__device__ __forceinline__ float pow2(int e)
{
    return __builtin_bit_cast(float, e > -127 ? (uint32_t)(e + 127) << 23 : 0x00400000u);
}

// Codes of 8 values over 2^e, the first in the low bits.
__device__ __forceinline__ uint32_t convert8(const float (&v)[8], int e)
{
    const float s = pow2(e);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}

__device__ __forceinline__ void put8(const Mx4RowArgs& a, int64_t row, int u, uint32_t w, int scale)
{
    ((uint32_t*)a.codes)[row * a.nb * 4 + u] = w;
    if ((u & 3) == 0) a.scale[row * a.nb + (u >> 2)] = (uint8_t)scale;
}

// One unit of 8 values of a row that is not normalised.
__device__ __forceinline__ void emit(const Mx4RowArgs& a, int64_t row, int u, const float (&x)[8])
{
    const float m = quad_max(max8(x));
    const bool odd = !(m <= 0x1.fffffep127f);  // NaN or infinity
    // frexp's exponent is one more than floor(log2 m), for subnormals too
    const int e = m == 0.0f || odd ? 0 : clamp_exp(__builtin_amdgcn_frexp_expf(m) - 3);
    put8(a, row, u, convert8(x, e), odd ? kNanScale : e + 127);
}

// What a normalised row's codes need beside its values.
struct Norm {
    double n;   // the norm
    float r;    // 1 / n
    bool zero;  // a row of zeros
    bool odd;   // holds a NaN or an infinity
    bool far;   // r may be subnormal or infinite: float64 throughout
};
__device__ __forceinline__ Norm norm_of(double ss, float top)
{
    Norm s;
    s.odd = !(top <= 0x1.fffffep127f);
    s.zero = !s.odd && top < kTiny;
    s.n = s.zero ? 1.0 : __builtin_sqrt(ss);
    s.r = (float)(1.0 / s.n);
    s.far = !(s.n > 0x1p-100 && s.n < 0x1p100);
    return s;
}

// The border between codes lies at magnitudes whose fraction is a multiple of a
// quarter, as do the powers of two: is v within 4 units in the last place of one?
__device__ __forceinline__ bool near_border(float v)
{
    return ((__builtin_bit_cast(uint32_t, v) + 4u) & 0x1fffffu) < 8u;
}

__device__ __forceinline__ uint32_t code_of(double v, int e)
{
    const double m = __builtin_ldexp(__builtin_fabs(v), -e);
    const uint32_t c = (uint32_t)(m > 0.25) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0);
    return c | (__builtin_signbit(v) ? 8u : 0u);
}

__device__ __forceinline__ void emit_norm(const Mx4RowArgs& a, int64_t row, int u, const float (&x)[8], const Norm& s)
{
    const float m = quad_max(max8(x));
    float v[8];
    const float vm = m * s.r;
    bool slow = s.far;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = s.zero ? 0.0f : x[i] * s.r;
        slow |= near_border(v[i]) && v[i] != 0.0f;
    }
    // every lane of the block takes the same way here: vm is the block's
    const bool slow_scale = m != 0.0f && (s.far || vm < 0x1p-100f || near_border(vm));
    int e = s.zero || m == 0.0f ? 0 : clamp_exp(__builtin_amdgcn_frexp_expf(vm) - 3);
    if (slow_scale && !s.zero) {
        const double q = (double)m / s.n;
        e = clamp_exp((int)(__builtin_bit_cast(uint64_t, q) >> 52) - 1023 - 2);
    }
    uint32_t w = convert8(v, s.odd ? 0 : e);
    if ((slow || slow_scale) && !s.zero) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= code_of((double)x[i] / s.n, e) << (4 * i);
    }
    put8(a, row, u, w, s.odd ? kNanScale : e + 127);
}

template <int E, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quantize_mx4_kernel(Mx4RowArgs a)
{
    const int lanes = 1 << a.log2_lanes, lane = threadIdx.x & (lanes - 1), units = 4 * a.nb;
    const int rows = kThreads >> a.log2_lanes;
    for (int64_t row = (int64_t)blockIdx.x * rows + (threadIdx.x >> a.log2_lanes); row < a.T; row += (int64_t)gridDim.x * rows) {
        if (a.mask && !a.mask[row]) {
            for (int u = lane; u < units; u += lanes) put8(a, row, u, 0, kZeroScale);
            continue;
        }
        for (int u = lane; u < units; u += 2 * lanes) {
            float x[2][8];
            load8<E, WHOLE>(a.X, row, a.d, 8 * u, x[0]);
            const bool more = u + lanes < units;  // the same for a quad: both are multiples of 4
            if (more) load8<E, WHOLE>(a.X, row, a.d, 8 * (u + lanes), x[1]);
            emit(a, row, u, x[0]);
            if (more) emit(a, row, u + lanes, x[1]);
        }
    }
}

__device__ __forceinline__ double lanes_sum(double v, int lanes)
{
    for (int m = 1; m < lanes; m *= 2) v += __shfl_xor(v, m, 64);
    return v;
}
__device__ __forceinline__ float lanes_max(float v, int lanes)
{
    for (int m = 1; m < lanes; m *= 2) v = __builtin_elementwise_maximum(v, shfl_xor_f(v, m));
    return v;
}

// U units of 8 values a lane stay in registers (0: the row is read twice).
template <int E, bool WHOLE, int U>
__global__ __launch_bounds__(kThreads) void quantize_mx4_norm_kernel(Mx4RowArgs a)
{
    constexpr int kHeld = U > 0 ? U : 1;
    const int lanes = 1 << a.log2_lanes, lane = threadIdx.x & (lanes - 1), units = 4 * a.nb;
    const int rows = kThreads >> a.log2_lanes;
    for (int64_t row = (int64_t)blockIdx.x * rows + (threadIdx.x >> a.log2_lanes); row < a.T; row += (int64_t)gridDim.x * rows) {
        if (a.mask && !a.mask[row]) {
            for (int u = lane; u < units; u += lanes) put8(a, row, u, 0, kZeroScale);
            continue;
        }
        float x[kHeld][8];
        double ss = 0.0;
        float top = 0.0f;
        auto add = [&](const float (&v)[8]) {
            top = __builtin_elementwise_maximum(top, max8(v));
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)v[i], (double)v[i], ss);
        };
        if constexpr (U > 0) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (lane + j * lanes < units) load8<E, WHOLE>(a.X, row, a.d, 8 * (lane + j * lanes), x[j]);
                else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j][i] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) add(x[j]);
        } else {
#pragma unroll 4
            for (int u = lane; u < units; u += lanes) {
                load8<E, WHOLE>(a.X, row, a.d, 8 * u, x[0]);
                add(x[0]);
            }
        }
        const Norm s = norm_of(lanes_sum(ss, lanes), lanes_max(top, lanes));
        if constexpr (U > 0) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (lane + j * lanes < units) emit_norm(a, row, lane + j * lanes, x[j], s);
        } else {
            for (int u = lane; u < units; u += lanes) {
                load8<E, WHOLE>(a.X, row, a.d, 8 * u, x[0]);
                emit_norm(a, row, u, x[0], s);
            }
        }
    }
}

// 8 values c .. c + 7 of a row of d, those that exist.
template <int OUT, bool WHOLE>
__device__ __forceinline__ void store8(void* Y, int64_t row, int d, int c, const float (&y)[8])
{
    char* p = (char*)Y + (row * d + c) * elem_bytes<OUT>();
    if (!WHOLE && c + 8 > d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i >= d) continue;
            if constexpr (OUT == kF32) ((float*)p)[i] = y[i];
            else ((uint16_t*)p)[i] = (uint16_t)half_bits(OUT, y[i]);
        }
        return;
    }
    u32x4 w[OUT == kF32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (OUT == kF32) {
            w[0][i] = __builtin_bit_cast(uint32_t, y[i]);
            w[OUT == kF32 ? 1 : 0][i] = __builtin_bit_cast(uint32_t, y[4 + i]);
        } else {
            w[0][i] = half_pair<OUT>(y[2 * i], y[2 * i + 1]);
        }
    }
#pragma unroll
    for (int j = 0; j < (OUT == kF32 ? 2 : 1); ++j) {
        if constexpr (WHOLE) ((u32x4*)p)[j] = w[j];
        else ((u32x4_any*)p)[j] = w[j];
    }
}

template <int OUT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void dequantize_mx4_kernel(Mx4RowArgs a)
{
    const int lanes = 1 << a.log2_lanes, lane = threadIdx.x & (lanes - 1), units = (a.d + 7) / 8;
    const int rows = kThreads >> a.log2_lanes;
    for (int64_t row = (int64_t)blockIdx.x * rows + (threadIdx.x >> a.log2_lanes); row < a.T; row += (int64_t)gridDim.x * rows) {
#pragma unroll 2
        for (int u = lane; u < units; u += lanes) {
            const uint32_t w = ((const uint32_t*)a.codes)[row * a.nb * 4 + u];
            const int b = a.scale[row * a.nb + (u >> 2)];
            const float s = pow2(b == kNanScale ? 0 : b - 127);
            const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
            const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
            float y[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = b == kNanScale ? __builtin_nanf("") : y[i];
            store8<OUT, WHOLE>(a.Y, row, a.d, 8 * u, y);
        }
    }
}

// The lanes of a row: a power of two from 4 to 64 that leaves a lane about two units.
int lanes_for(int units)
{
    int l = 2;
    while (l < 6 && (2 << l) < units) ++l;
    return l;
}
dim3 row_grid(const Mx4RowArgs& a)
{
    const int64_t rows = kThreads >> a.log2_lanes, b = (a.T + rows - 1) / rows;
    return dim3((unsigned)(b < kMaxBlocks ? b : kMaxBlocks));
}

template <int E, bool WHOLE>
void quantize(const Mx4RowArgs& a, bool normalize, hipStream_t stream)
{
    const dim3 grid = row_grid(a), block(kThreads);
    const int per_lane = (4 * a.nb + (1 << a.log2_lanes) - 1) >> a.log2_lanes;
    if (!normalize) hipLaunchKernelGGL((quantize_mx4_kernel<E, WHOLE>), grid, block, 0, stream, a);
    else if (per_lane <= 2) hipLaunchKernelGGL((quantize_mx4_norm_kernel<E, WHOLE, 2>), grid, block, 0, stream, a);
    else if (per_lane <= 4) hipLaunchKernelGGL((quantize_mx4_norm_kernel<E, WHOLE, 4>), grid, block, 0, stream, a);
    else if (per_lane <= 8) hipLaunchKernelGGL((quantize_mx4_norm_kernel<E, WHOLE, 8>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((quantize_mx4_norm_kernel<E, WHOLE, 0>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_quantize_mx4(int elem, Mx4RowArgs a, bool normalize, hipStream_t stream)
{
    a.log2_lanes = lanes_for(4 * a.nb);
    const bool whole = a.d % 8 == 0;
    // rows of 16-bit values of which 8 divide the width are 16-byte aligned, as are those of 32-bit ones
#define MAXSIM_MX4_TYPE(E) (whole ? quantize<E, true>(a, normalize, stream) : quantize<E, false>(a, normalize, stream))
    if (elem == kF32) MAXSIM_MX4_TYPE(kF32);
    else if (elem == kBF16) MAXSIM_MX4_TYPE(kBF16);
    else MAXSIM_MX4_TYPE(kF16);
#undef MAXSIM_MX4_TYPE
    return hipGetLastError();
}

hipError_t launch_dequantize_mx4(Mx4RowArgs a, hipStream_t stream)
{
    a.log2_lanes = lanes_for((a.d + 7) / 8);
    const dim3 grid = row_grid(a), block(kThreads);
    const bool whole = a.d % 8 == 0;
#define MAXSIM_MX4_TYPE(E)                                                                                  \
    do {                                                                                                    \
        if (whole) hipLaunchKernelGGL((dequantize_mx4_kernel<E, true>), grid, block, 0, stream, a);          \
        else hipLaunchKernelGGL((dequantize_mx4_kernel<E, false>), grid, block, 0, stream, a);               \
    } while (0)
    if (a.out == kF32) MAXSIM_MX4_TYPE(kF32);
    else if (a.out == kBF16) MAXSIM_MX4_TYPE(kBF16);
    else MAXSIM_MX4_TYPE(kF16);
#undef MAXSIM_MX4_TYPE
    return hipGetLastError();
}

}  // namespace maxsim
