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
// With normalisation the row stays in registers while its squares are summed. A code
// is decided on the quotient x / ||x||, and one that falls on the wrong side of a
// border is a whole step off. So the float32 quotient is used only where it is
// further from every border than its error can be; a wave that holds another one
// (one in about 50) sums the squares again in float64 and forms those in float64.
//
// 360,000 rows of 128 fp16 values, a quarter masked, normalised: 27.5 us for 94 MB
// (38.6 us with every quotient in float64), and 32.5 us for the 209 MB of the way back
// to float32; one query's 32 rows of 768 3.2 us each way, which is a launch.
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

// The code of v / 2^e, v not NaN.
__device__ __forceinline__ uint32_t code_of(double v, int e)
{
    const double m = __builtin_ldexp(__builtin_fabs(v), -e);
    const uint32_t c = (uint32_t)(m > 0.25) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0);
    return c | (__builtin_signbit(v) ? 8u : 0u);
}
// The exponent of a block of largest magnitude m > 0 over the norm n.
__device__ __forceinline__ int exact_exp(double n, float m)
{
    return clamp_exp((int)(__builtin_bit_cast(uint64_t, (double)m / n) >> 52) - 1023 - 2);
}

// The borders between codes lie at magnitudes whose fraction is a multiple of a
// quarter, as do the powers of two: a number below 2 W << 11 where v is within W
// units in the last place of one.
template <int W>
__device__ __forceinline__ uint32_t from_border(float v)
{
    return (__builtin_bit_cast(uint32_t, v) + (uint32_t)W) << 11;
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

// Sum or maximum over the G lanes of a row, the same bits in every lane.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <int G, typename OP>
__device__ __forceinline__ float lanes_reduce(float v, OP op)
{
    v = op(v, dpp_f<0xB1>(v));  // quad_perm [1,0,3,2]
    v = op(v, dpp_f<0x4E>(v));  // quad_perm [2,3,0,1]
    if constexpr (G >= 8) v = op(v, dpp_f<0x141>(v));   // row_half_mirror
    if constexpr (G >= 16) v = op(v, dpp_f<0x140>(v));  // row_mirror
    if constexpr (G >= 32) v = op(v, shfl_xor_f(v, 16));
    if constexpr (G >= 64) v = op(v, shfl_xor_f(v, 32));
    return v;
}
template <int G>
__device__ __forceinline__ double lanes_sum(double v)
{
#pragma unroll
    for (int m = 1; m < G; m *= 2) v += __shfl_xor(v, m, 64);
    return v;
}

// G lanes hold a row, U units of 8 values each.
template <int E, bool WHOLE, int G, int U>
__global__ __launch_bounds__(kThreads) void quantize_mx4_norm_kernel(Mx4RowArgs a)
{
    // A square passes 2 U + 8 additions (four sums in a lane, 64 lanes at most), each off
    // by 2^-24 of the sum, and the root by half of that; the root, its reciprocal and
    // the product add less than 4 units. A unit in the last place is at least 2^-24 of
    // the value.
    constexpr int W = U + 12;
    const int lane = threadIdx.x & (G - 1), units = 4 * a.nb;
    constexpr int rows = kThreads / G;
    for (int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / G; row < a.T; row += (int64_t)gridDim.x * rows) {
        const bool live = !a.mask || a.mask[row];
        if (!__any(live)) {  // the end of a padded document
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (lane + j * G < units) put8(a, row, lane + j * G, 0, kZeroScale);
            continue;
        }
        float x[U][8], part[4] = {0.0f, 0.0f, 0.0f, 0.0f}, top = 0.0f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (live && lane + j * G < units) load8<E, WHOLE>(a.X, row, a.d, 8 * (lane + j * G), x[j]);
            else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = 0.0f;
            }
        }
        float m[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            m[j] = quad_max(max8(x[j]));
            top = __builtin_elementwise_maximum(top, m[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i & 3] = __builtin_fmaf(x[j][i], x[j][i], part[i & 3]);
        }
        const float ss = lanes_reduce<G>((part[0] + part[1]) + (part[2] + part[3]), [](float p, float q) { return p + q; });
        top = lanes_reduce<G>(top, [](float p, float q) { return __builtin_elementwise_maximum(p, q); });
        const bool odd = !(top <= 0x1.fffffep127f), zero = !odd && top < kTiny;
        const bool far = !zero && !odd && !(ss > 0x1p-100f && ss < 0x1p100f);
        const float r = zero || far ? 0.0f : rsqrt_f(ss);
        constexpr uint32_t kNear = (uint32_t)(2 * W) << 11;
        uint32_t w[U], near = 0xffffffffu;
        int e[U];
        bool small = far;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float v[8];
            uint32_t least = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = x[j][i] * r;
                const uint32_t b = from_border<W>(v[i]);
                least = b < least ? b : least;
            }
            if (least < kNear) {  // zeros look like borders
                least = 0xffffffffu;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t b = v[i] != 0.0f ? from_border<W>(v[i]) : 0xffffffffu;
                    least = b < least ? b : least;
                }
            }
            near = least < near ? least : near;
            const float vm = m[j] * r;
            // frexp's exponent of 0 is 0 too: blocks of zeros have e = 0
            e[j] = vm == 0.0f ? 0 : clamp_exp(__builtin_amdgcn_frexp_expf(vm) - 3);
            w[j] = convert8(v, e[j]);
            small |= vm < 0x1p-100f && m[j] != 0.0f;
        }
        if (__any((near < kNear || small) && !zero && !odd)) {
            // the row is read again, so that it need not stay in registers until here
            auto again = [&](int j, float (&y)[8]) {
                const int u = lane + j * G;
                load8<E, WHOLE>(a.X, row, a.d, u < units ? 8 * u : 0, y);
                if (!live || u >= units) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
                }
            };
            double s64 = 0.0;
#pragma unroll 1
            for (int j = 0; j < U; ++j) {
                float y[8];
                again(j, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) s64 = __builtin_fma((double)y[i], (double)y[i], s64);
            }
            const double n = __builtin_sqrt(lanes_sum<G>(s64));
#pragma unroll
            for (int j = 0; j < U; ++j) {
                float y[8];
                again(j, y);
                // a block's exponent is formed again in all its lanes or in none, with all its
                // codes; otherwise single codes are
                const float m = quad_max(max8(y));
                const bool some = m != 0.0f && !zero && !odd, all = some && (small || from_border<W>(m * r) < kNear);
                if (all) e[j] = exact_exp(n, m);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (all || (some && from_border<W>(y[i] * r) < kNear && y[i] != 0.0f))
                        w[j] = (w[j] & ~(15u << (4 * i))) | code_of((double)y[i] / n, e[j]) << (4 * i);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (lane + j * G < units) put8(a, row, lane + j * G, w[j], odd ? kNanScale : e[j] + 127);
    }
}

// Rows longer than the registers hold: one wave per row, read twice, in float64
// throughout.
template <int E, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quantize_mx4_norm_long_kernel(Mx4RowArgs a)
{
    const int lane = threadIdx.x & 63, units = 4 * a.nb;
    constexpr int rows = kThreads / 64;
    for (int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / 64; row < a.T; row += (int64_t)gridDim.x * rows) {
        if (a.mask && !a.mask[row]) {
            for (int u = lane; u < units; u += 64) put8(a, row, u, 0, kZeroScale);
            continue;
        }
        float x[8], top = 0.0f;
        double ss = 0.0;
#pragma unroll 4
        for (int u = lane; u < units; u += 64) {
            load8<E, WHOLE>(a.X, row, a.d, 8 * u, x);
            top = __builtin_elementwise_maximum(top, max8(x));
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)x[i], (double)x[i], ss);
        }
        top = lanes_reduce<64>(top, [](float p, float q) { return __builtin_elementwise_maximum(p, q); });
        const double n = __builtin_sqrt(lanes_sum<64>(ss));
        const bool odd = !(top <= 0x1.fffffep127f), zero = !odd && top < kTiny;
        for (int u = lane; u < units; u += 64) {
            load8<E, WHOLE>(a.X, row, a.d, 8 * u, x);
            const float m = quad_max(max8(x));
            int e = 0;
            uint32_t w = 0;
            if (!odd && !zero && m != 0.0f) {
                e = exact_exp(n, m);
#pragma unroll
                for (int i = 0; i < 8; ++i) w |= code_of((double)x[i] / n, e) << (4 * i);
            } else {  // zeros, which keep their signs (or a row marked NaN: any codes)
#pragma unroll
                for (int i = 0; i < 8; ++i) w |= (__builtin_bit_cast(uint32_t, x[i]) >> 31) << (4 * i + 3);
            }
            put8(a, row, u, w, odd ? kNanScale : e + 127);
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
    const int units = 4 * a.nb;
#define MAXSIM_MX4_NORM(G, U) hipLaunchKernelGGL((quantize_mx4_norm_kernel<E, WHOLE, G, U>), grid, block, 0, stream, a)
    if (!normalize) hipLaunchKernelGGL((quantize_mx4_kernel<E, WHOLE>), grid, block, 0, stream, a);
    else if (units <= 8) MAXSIM_MX4_NORM(4, 2);
    else if (units <= 16) MAXSIM_MX4_NORM(8, 2);
    else if (units <= 32) MAXSIM_MX4_NORM(16, 2);
    else if (units <= 64) MAXSIM_MX4_NORM(32, 2);
    else if (units <= 128) MAXSIM_MX4_NORM(64, 2);
    else if (units <= 256) MAXSIM_MX4_NORM(64, 4);
    else if (units <= 512) MAXSIM_MX4_NORM(64, 8);
    else if (units <= 1024) MAXSIM_MX4_NORM(64, 16);
    else hipLaunchKernelGGL((quantize_mx4_norm_long_kernel<E, WHOLE>), grid, block, 0, stream, a);
#undef MAXSIM_MX4_NORM
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
