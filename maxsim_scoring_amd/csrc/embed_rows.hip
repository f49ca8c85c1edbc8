// Row operators of the embedding head for gfx950: token quantisation, row
// normalisation and its gradient, and dropout from a counter-based generator.
//
// All of them are bound by memory: a row is read once, kept in registers while
// its statistics are reduced over the lanes that hold it, and its outputs are
// written once. G lanes (4 to 64) share a row, so that narrow rows fill whole
// waves and a reduction takes log2(G) cross-lane steps; each lane holds VPL
// chunks of VB bytes. Rows too long for that are read twice (the second time
// from the L2). Measured: codes of 360,000 x 128 fp16 rows, a quarter of them
// masked, in 21.4 to 23.6 us (5.0 to 5.5 TB/s; a copy reaches 5.4), 131,072 x 128
// bf16 rows normalised in 11.0 us (5.4 TB/s), their gradient in 23.3 (5.8 TB/s).
// Rows that 16 bytes do not divide go element by element: 131,072 rows of 100 bf16
// values take 27 us to codes, 27 normalised, 35 in the gradient; of 128 values
// 11.7, 11.9 and 23.4.
#include "embed_common.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 22;  // blocks x threads stays far below 2^32

template <int E> constexpr int elem_bytes() { return E == kF32 ? 4 : 2; }

// One chunk of VB bytes (16, or a single element) of a row.
template <int VB> struct Raw;
template <> struct Raw<16> { typedef u32x4 T; };
template <> struct Raw<4> { typedef uint32_t T; };
template <> struct Raw<2> { typedef uint16_t T; };

template <int E>
__device__ __forceinline__ float to_float(uint32_t bits)
{
    if constexpr (E == kF32) return __builtin_bit_cast(float, bits);
    else if constexpr (E == kBF16) return __builtin_bit_cast(float, bits << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

template <int E, int VB>
__device__ __forceinline__ void unpack(typename Raw<VB>::T raw, float (&x)[VB / elem_bytes<E>()])
{
    if constexpr (VB == 16 && E == kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = to_float<E>(raw[i]);
    } else if constexpr (VB == 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = to_float<E>(raw[i] & 0xffffu);
            x[2 * i + 1] = E == kBF16 ? __builtin_bit_cast(float, raw[i] & 0xffff0000u) : to_float<E>(raw[i] >> 16);
        }
    } else {
        x[0] = to_float<E>((uint32_t)raw);
    }
}

// C values to element `at` of Y (type `out`, uniform); at is a multiple of C.
template <int C>
__device__ __forceinline__ void store(void* Y, int out, int64_t at, const float (&y)[C])
{
    if (out == kF32) {
        float* p = (float*)Y + at;
        if constexpr (C == 1) p[0] = y[0];
        else {
#pragma unroll
            for (int i = 0; i < C / 4; ++i)
                ((f32x4*)p)[i] = f32x4{y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
        }
        return;
    }
    uint16_t* p = (uint16_t*)Y + at;
    if constexpr (C == 1) p[0] = (uint16_t)half_bits(out, y[0]);
    else {
        uint32_t w[C / 2];
        if (out == kBF16) {
#pragma unroll
            for (int i = 0; i < C / 2; ++i) w[i] = half_pair<kBF16>(y[2 * i], y[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < C / 2; ++i) w[i] = half_pair<kF16>(y[2 * i], y[2 * i + 1]);
        }
        if constexpr (C == 8) *(u32x4*)p = u32x4{w[0], w[1], w[2], w[3]};
        else *(u32x2*)p = u32x2{w[0], w[1]};
    }
}

// Sum or max over the G lanes of a row group, the same bits in every lane.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
template <int G, typename OP>
__device__ __forceinline__ float group_reduce(float v, OP op)
{
    static_assert(G == 4 || G == 8 || G == 16 || G == 32 || G == 64, "lanes per row");
    v = op(v, dpp_f<0xB1>(v));  // quad_perm [1,0,3,2]
    v = op(v, dpp_f<0x4E>(v));  // quad_perm [2,3,0,1]
    if constexpr (G >= 8) v = op(v, dpp_f<0x141>(v));   // row_half_mirror
    if constexpr (G >= 16) v = op(v, dpp_f<0x140>(v));  // row_mirror
    if constexpr (G >= 32) v = op(v, shfl_xor_f(v, 16));
    if constexpr (G >= 64) v = op(v, shfl_xor_f(v, 32));
    return v;
}
struct Add { __device__ __forceinline__ float operator()(float a, float b) const { return a + b; } };
struct Max { __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); } };
// The maximum that is NaN where either operand is (v_maximum3_f32).
struct MaxNan { __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_elementwise_maximum(a, b); } };

// ---------------------------------------------------------------------------
// Quantisation
// ---------------------------------------------------------------------------

// What the codes of a row need beside its values.
struct Quant {
    float top;   // largest magnitude
    float inv;   // about 127 / top; 0 where every code is decided in float64
    float near;  // how far from an integer a code is decided in float64, -1: always, 1: never
    bool zero;
};
__device__ __forceinline__ Quant quant_of(float top)
{
    Quant s;
    s.top = top;
    s.zero = top < kTiny;
    const bool large = !(top < 0x1p120f);  // the reciprocal vanishes from 2^126 on
    s.inv = s.zero || large ? 0.0f : 127.0f * __builtin_amdgcn_rcpf(top);
    // a NaN or an infinity leaves the codes open; the scale comes out as NaN
    s.near = !large ? 0.5f - 0x1p-14f : top <= 0x1.fffffep127f ? -1.0f : 1.0f;
    return s;
}

// Codes of C values of a row; adds the squares of 127 x / top to ss.
//
// v = x * inv is within 127 * 2^-22 = 2^-15 of 127 x / top (the reciprocal is
// off by 2^-23 relative, two products by 2^-24 each). So the nearest integer to
// v is the nearest to the quotient unless v is that close to the middle between
// two integers; then the quotient is formed in float64. There it is a fraction
// of two numbers of 31 and 24 bits: it is exactly a half, or further from one
// than 2^-26, so a correctly rounded division (2^-46) decides it. The slow
// branch is taken for about one chunk of 8 in 1,000.
template <int C, bool SQUARES>
__device__ __forceinline__ void make_codes(const float (&x)[C], const Quant& s, float& ss, uint32_t (&w)[(C + 3) / 4])
{
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: the sum's low bits are the integer, ties to even
    uint32_t b[C];
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const float v = x[i] * s.inv;
        const float m = v + kMagic;
        b[i] = __builtin_bit_cast(uint32_t, m);
        off = __builtin_fmaxf(off, __builtin_fabsf(v - (m - kMagic)));
        if (SQUARES) ss = __builtin_fmaf(v, v, ss);
    }
    if (off >= s.near) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            b[i] = (uint32_t)(int)__builtin_rint((double)x[i] * 127.0 / (double)s.top);
        if (SQUARES && s.near < 0.0f) {  // the values above were x * 0
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float v = (float)((double)x[i] * 127.0 / (double)s.top);
                ss = __builtin_fmaf(v, v, ss);
            }
        }
    }
    if constexpr (C == 1) {
        w[0] = b[0];
    } else {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
            const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x0c0c0400u);
            w[i] = lo | hi << 16;
        }
    }
}

template <int C>
__device__ __forceinline__ void store_codes(void* Y, int64_t at, const uint32_t (&w)[(C + 3) / 4])
{
    int8_t* p = (int8_t*)Y + at;
    if constexpr (C == 1) p[0] = (int8_t)w[0];
    else if constexpr (C == 4) *(uint32_t*)p = w[0];
    else *(u32x2*)p = u32x2{w[0], w[1]};
}

// top / 127: the product with 1/127 and one correction step; or 1 / sqrt(ss).
// Both are NaN where the row holds a NaN (top and ss are) or an infinity (top is
// one, and x * inv is Inf * 0).
__device__ __forceinline__ float quant_scale(const Quant& s, bool normalize, float ss)
{
    if (s.zero) return 1.0f;
    if (normalize) return rsqrt_f(ss);
    const float q = s.top * (1.0f / 127.0f);
    return __builtin_fmaf(__builtin_fmaf(-q, 127.0f, s.top), 1.0f / 127.0f, q);
}

template <int E, int VB, int G, int VPL, bool NORM>
__device__ __forceinline__ void quantize_rows(const RowArgs& a)
{
    constexpr int C = VB / elem_bytes<E>();
    typedef typename Raw<VB>::T R;
    const int lane = threadIdx.x % G;
    const int nv = a.d / C;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.T;
         row += (int64_t)gridDim.x * (kThreads / G)) {
        const bool live = !a.mask || a.mask[row];
        const R* src = (const R*)a.X + row * nv;
        R raw[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) raw[j] = live && lane + j * G < nv ? src[lane + j * G] : R{};
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float x[C];
            unpack<E, VB>(raw[j], x);
#pragma unroll
            for (int i = 0; i < C; ++i) top = MaxNan{}(top, __builtin_fabsf(x[i]));
        }
        const Quant s = quant_of(group_reduce<G>(top, MaxNan{}));
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float x[C];
            uint32_t w[(C + 3) / 4];
            unpack<E, VB>(raw[j], x);
            make_codes<C, NORM>(x, s, ss, w);
            if (lane + j * G < nv) store_codes<C>(a.Y, row * a.d + (int64_t)(lane + j * G) * C, w);
        }
        if (NORM) ss = group_reduce<G>(ss, Add{});
        if (lane == 0) a.stat[row] = quant_scale(s, NORM, ss);
    }
}
template <int E, int VB, int G, int VPL>
__global__ __launch_bounds__(kThreads) void quantize_kernel(RowArgs a)
{
    if (a.normalize) quantize_rows<E, VB, G, VPL, true>(a);
    else quantize_rows<E, VB, G, VPL, false>(a);
}

// Rows longer than the register forms hold: one wave per row, read twice.
template <int E, int VB>
__global__ __launch_bounds__(kThreads) void quantize_long_kernel(RowArgs a)
{
    constexpr int C = VB / elem_bytes<E>();
    typedef typename Raw<VB>::T R;
    const int lane = threadIdx.x % 64;
    const int nv = a.d / C;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64; row < a.T;
         row += (int64_t)gridDim.x * (kThreads / 64)) {
        const bool live = !a.mask || a.mask[row];
        const R* src = (const R*)a.X + row * nv;
        float top = 0.0f;
        if (live) {
#pragma unroll 8
            for (int c = lane; c < nv; c += 64) {
                float x[C];
                unpack<E, VB>(src[c], x);
#pragma unroll
                for (int i = 0; i < C; ++i) top = MaxNan{}(top, __builtin_fabsf(x[i]));
            }
        }
        const Quant s = quant_of(group_reduce<64>(top, MaxNan{}));
        float ss = 0.0f;
#pragma unroll 4
        for (int c = lane; c < nv; c += 64) {
            float x[C];
            uint32_t w[(C + 3) / 4];
            unpack<E, VB>(live ? src[c] : R{}, x);
            make_codes<C, true>(x, s, ss, w);
            store_codes<C>(a.Y, row * a.d + (int64_t)c * C, w);
        }
        ss = group_reduce<64>(ss, Add{});
        if (lane == 0) a.stat[row] = quant_scale(s, a.normalize != 0, ss);
    }
}

// ---------------------------------------------------------------------------
// Normalisation
// ---------------------------------------------------------------------------

// The norm's reciprocal as two factors, 1 / ||x|| = r * s, from the row's
// largest magnitude and sum of squares: s is 1 while the sum of squares neither
// overflows nor loses its small terms; otherwise the sum of squares has to be
// that of the row divided by top, and s = 1 / top.
constexpr float kSumLow = 0x1p-100f, kSumHigh = 0x1p126f;

template <int E, int VB, int G, int VPL>
__global__ __launch_bounds__(kThreads) void normalize_fwd_kernel(RowArgs a)
{
    constexpr int C = VB / elem_bytes<E>();
    typedef typename Raw<VB>::T R;
    const int lane = threadIdx.x % G;
    const int nv = a.d / C;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.T;
         row += (int64_t)gridDim.x * (kThreads / G)) {
        const bool live = !a.mask || a.mask[row];
        const R* src = (const R*)a.X + row * nv;
        R raw[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) raw[j] = live && lane + j * G < nv ? src[lane + j * G] : R{};
        float top = 0.0f, ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float x[C];
            unpack<E, VB>(raw[j], x);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                top = __builtin_fmaxf(top, __builtin_fabsf(x[i]));
                ss = __builtin_fmaf(x[i], x[i], ss);
            }
        }
        top = group_reduce<G>(top, Max{});
        ss = group_reduce<G>(ss, Add{});
        float s = 1.0f;
        const bool zero = top < kTiny && !(ss != ss);
        if (!zero && !(ss >= kSumLow && ss <= kSumHigh)) {
            s = 1.0f / top;
            ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                float x[C];
                unpack<E, VB>(raw[j], x);
#pragma unroll
                for (int i = 0; i < C; ++i) ss = __builtin_fmaf(x[i] * s, x[i] * s, ss);
            }
            ss = group_reduce<G>(ss, Add{});
        }
        const float r = rsqrt_f(ss);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float x[C];
            unpack<E, VB>(raw[j], x);
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = zero ? 0.0f : x[i] * s * r;
            if (lane + j * G < nv) store<C>(a.Y, a.out, row * a.d + (int64_t)(lane + j * G) * C, x);
        }
        if (lane == 0) a.stat[row] = zero ? 0.0f : r * s;
    }
}

template <int E, int VB>
__global__ __launch_bounds__(kThreads) void normalize_fwd_long_kernel(RowArgs a)
{
    constexpr int C = VB / elem_bytes<E>();
    typedef typename Raw<VB>::T R;
    const int lane = threadIdx.x % 64;
    const int nv = a.d / C;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64; row < a.T;
         row += (int64_t)gridDim.x * (kThreads / 64)) {
        const bool live = !a.mask || a.mask[row];
        const R* src = (const R*)a.X + row * nv;
        float top = 0.0f, ss = 0.0f;
        if (live) {
#pragma unroll 8
            for (int c = lane; c < nv; c += 64) {
                float x[C];
                unpack<E, VB>(src[c], x);
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    top = __builtin_fmaxf(top, __builtin_fabsf(x[i]));
                    ss = __builtin_fmaf(x[i], x[i], ss);
                }
            }
        }
        top = group_reduce<64>(top, Max{});
        ss = group_reduce<64>(ss, Add{});
        float s = 1.0f;
        const bool zero = top < kTiny && !(ss != ss);
        if (!zero && !(ss >= kSumLow && ss <= kSumHigh)) {
            s = 1.0f / top;
            ss = 0.0f;
            for (int c = lane; c < nv; c += 64) {
                float x[C];
                unpack<E, VB>(src[c], x);
#pragma unroll
                for (int i = 0; i < C; ++i) ss = __builtin_fmaf(x[i] * s, x[i] * s, ss);
            }
            ss = group_reduce<64>(ss, Add{});
        }
        const float r = rsqrt_f(ss);
#pragma unroll 4
        for (int c = lane; c < nv; c += 64) {
            float x[C];
            unpack<E, VB>(zero ? R{} : src[c], x);
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = zero ? 0.0f : x[i] * s * r;
            store<C>(a.Y, a.out, row * a.d + (int64_t)c * C, x);
        }
        if (lane == 0) a.stat[row] = zero ? 0.0f : r * s;
    }
}

template <int C>
__device__ __forceinline__ void load_grad(const float* g, float (&y)[C])
{
    if constexpr (C == 1) y[0] = g[0];
    else {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
            const f32x4 v = ((const f32x4*)g)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[4 * i + k] = v[k];
        }
    }
}

// dx = rnorm (g - u <u, g>), u = x rnorm
template <int E, int VB, int G, int VPL>
__global__ __launch_bounds__(kThreads) void normalize_bwd_kernel(RowArgs a)
{
    constexpr int C = VB / elem_bytes<E>();
    typedef typename Raw<VB>::T R;
    const int lane = threadIdx.x % G;
    const int nv = a.d / C;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.T;
         row += (int64_t)gridDim.x * (kThreads / G)) {
        const float rn = a.rnorm[row];
        const bool live = rn != 0.0f;
        const R* src = (const R*)a.X + row * nv;
        const float* up = a.g + row * a.d;
        R raw[VPL];
        float g[VPL][C];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const bool in = live && lane + j * G < nv;
            raw[j] = in ? src[lane + j * G] : R{};
            if (in) load_grad<C>(up + (lane + j * G) * C, g[j]);
            else {
#pragma unroll
                for (int i = 0; i < C; ++i) g[j][i] = 0.0f;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float x[C];
            unpack<E, VB>(raw[j], x);
#pragma unroll
            for (int i = 0; i < C; ++i) dot = __builtin_fmaf(x[i] * rn, g[j][i], dot);
        }
        dot = group_reduce<G>(dot, Add{});
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float x[C];
            unpack<E, VB>(raw[j], x);
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = live ? rn * (g[j][i] - x[i] * rn * dot) : 0.0f;
            if (lane + j * G < nv) store<C>(a.Y, a.out, row * a.d + (int64_t)(lane + j * G) * C, x);
        }
    }
}

template <int E, int VB>
__global__ __launch_bounds__(kThreads) void normalize_bwd_long_kernel(RowArgs a)
{
    constexpr int C = VB / elem_bytes<E>();
    typedef typename Raw<VB>::T R;
    const int lane = threadIdx.x % 64;
    const int nv = a.d / C;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64; row < a.T;
         row += (int64_t)gridDim.x * (kThreads / 64)) {
        const float rn = a.rnorm[row];
        const bool live = rn != 0.0f;
        const R* src = (const R*)a.X + row * nv;
        const float* up = a.g + row * a.d;
        float dot = 0.0f;
        if (live) {
#pragma unroll 4
            for (int c = lane; c < nv; c += 64) {
                float x[C], g[C];
                unpack<E, VB>(src[c], x);
                load_grad<C>(up + (int64_t)c * C, g);
#pragma unroll
                for (int i = 0; i < C; ++i) dot = __builtin_fmaf(x[i] * rn, g[i], dot);
            }
        }
        dot = group_reduce<64>(dot, Add{});
#pragma unroll 4
        for (int c = lane; c < nv; c += 64) {
            float x[C] = {}, g[C] = {};
            if (live) {
                unpack<E, VB>(src[c], x);
                load_grad<C>(up + (int64_t)c * C, g);
            }
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = live ? rn * (g[i] - x[i] * rn * dot) : 0.0f;
            store<C>(a.Y, a.out, row * a.d + (int64_t)c * C, x);
        }
    }
}

// ---------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products.
// One call gives 128 bits, 16 for each of 8 elements: with 32 bits for each,
// the products would take longer than the memory traffic of 16-bit tensors.
__device__ __forceinline__ u32x4 philox(uint64_t index, uint64_t step, uint32_t k0, uint32_t k1)
{
    uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32);
    uint32_t c2 = (uint32_t)step, c3 = (uint32_t)(step >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0;
        const uint64_t p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// One group of 8 elements per thread: with the next group's loads issued ahead in
// the same thread, 100 million bf16 values took 75.6 us (two groups) and 72.9 us
// (four), with one 67.6 us (5.96 TB/s, where a plain copy of them reaches 5.4).
template <int E>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropArgs a)
{
    constexpr int NR = E == kF32 ? 2 : 1;  // 16-byte chunks of 8 elements
    constexpr int C = 16 / elem_bytes<E>();
    const uint64_t step = a.step + (a.step_dev ? *a.step_dev : 0);
    const int64_t full = a.n / 8;  // whole groups
    for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g * 8 < a.n; g += (int64_t)gridDim.x * kThreads) {
        u32x4 raw[NR];
#pragma unroll
        for (int h = 0; h < NR; ++h) raw[h] = g < full ? ((const u32x4*)a.X)[g * NR + h] : u32x4{};
        const u32x4 w = philox((uint64_t)g, step, a.seed_lo, a.seed_hi);
        if (g < full) {
#pragma unroll
            for (int h = 0; h < NR; ++h) {
                float x[C];
                unpack<E, 16>(raw[h], x);
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int e = h * C + i;
                    const uint32_t bits = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
                    x[i] = bits < a.q ? 0.0f : x[i] * a.up;
                }
                store<C>(a.Y, E, g * 8 + h * C, x);
            }
        } else {
            // the elements behind the last whole group
            typedef typename Raw<elem_bytes<E>()>::T R;
            for (int e = 0; e < (int)(a.n - full * 8); ++e) {
                float x[1];
                unpack<E, elem_bytes<E>()>(((const R*)a.X)[g * 8 + e], x);
                const uint32_t word = e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3];
                const uint32_t bits = e & 1 ? word >> 16 : word & 0xffffu;
                x[0] = bits < a.q ? 0.0f : x[0] * a.up;
                store<1>(a.Y, E, g * 8 + e, x);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

unsigned row_blocks(int64_t T, int rows)
{
    const int64_t b = (T + rows - 1) / rows;
    return (unsigned)(b < kMaxBlocks ? b : kMaxBlocks);
}

// Picks the lanes per row and chunks per lane from the number of chunks; V
// chunks per lane in the narrow classes. Quantisation's work per row (its
// reduction, reciprocal and scale) is as long as that of a chunk, so two chunks
// share it: 360,000 rows of 128 fp16 values take 21.5 us with 8 lanes x 2 chunks,
// 43 with 16 x 1 and 23.7 with 4 x 4; normalisation of 131,072 such rows 10.9,
// 11.3 and 10.9 us; its gradient, with 48 bytes to load per chunk, 23.8, 23.0
// and 24.2 us.
#define MAXSIM_ROWS(KERNEL, LONG, E, VB, V, MAXV)                                                            \
    do {                                                                                                     \
        const int nv = a.d / (VB / elem_bytes<E>());                                                          \
        if (nv <= 8) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 8 / V, V);                                              \
        else if (nv <= 16) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 16 / V, V);                                       \
        else if (nv <= 32) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 32 / V, V);                                       \
        else if (nv <= 64) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 64 / V, V);                                       \
        else if (nv <= 128) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 64, 2);                                          \
        else if (nv <= 256) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 64, 4);                                          \
        else if (nv <= 512) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 64, 8);                                          \
        else if (MAXV >= 16 && nv <= 1024) MAXSIM_ROW_LAUNCH(KERNEL, E, VB, 64, (MAXV >= 16 ? 16 : 8));      \
        else hipLaunchKernelGGL((LONG<E, VB>), dim3(row_blocks(a.T, kThreads / 64)), dim3(kThreads), 0, stream, a); \
    } while (0)
#define MAXSIM_ROW_LAUNCH(KERNEL, E, VB, G, VPL) \
    hipLaunchKernelGGL((KERNEL<E, VB, G, VPL>), dim3(row_blocks(a.T, kThreads / (G))), dim3(kThreads), 0, stream, a)
#define MAXSIM_ROW_TYPES(KERNEL, LONG, V, MAXV)                                          \
    do {                                                                                 \
        if (elem == kF32) {                                                              \
            if (a.d % 4 == 0) MAXSIM_ROWS(KERNEL, LONG, kF32, 16, V, MAXV);                 \
            else MAXSIM_ROWS(KERNEL, LONG, kF32, 4, V, MAXV);                               \
        } else if (elem == kBF16) {                                                      \
            if (a.d % 8 == 0) MAXSIM_ROWS(KERNEL, LONG, kBF16, 16, V, MAXV);                \
            else MAXSIM_ROWS(KERNEL, LONG, kBF16, 2, V, MAXV);                              \
        } else {                                                                         \
            if (a.d % 8 == 0) MAXSIM_ROWS(KERNEL, LONG, kF16, 16, V, MAXV);                 \
            else MAXSIM_ROWS(KERNEL, LONG, kF16, 2, V, MAXV);                               \
        }                                                                                \
    } while (0)

}  // namespace

hipError_t launch_quantize(int elem, RowArgs a, hipStream_t stream)
{
    MAXSIM_ROW_TYPES(quantize_kernel, quantize_long_kernel, 2, 16);
    return hipGetLastError();
}

hipError_t launch_normalize_fwd(int elem, RowArgs a, hipStream_t stream)
{
    MAXSIM_ROW_TYPES(normalize_fwd_kernel, normalize_fwd_long_kernel, 2, 16);
    return hipGetLastError();
}

hipError_t launch_normalize_bwd(int elem, RowArgs a, hipStream_t stream)
{
    MAXSIM_ROW_TYPES(normalize_bwd_kernel, normalize_bwd_long_kernel, 1, 8);
    return hipGetLastError();
}

hipError_t launch_dropout(int elem, DropArgs a, hipStream_t stream)
{
    const dim3 grid(row_blocks((a.n + 7) / 8, kThreads)), block(kThreads);
    if (elem == kF32) hipLaunchKernelGGL((dropout_kernel<kF32>), grid, block, 0, stream, a);
    else if (elem == kBF16) hipLaunchKernelGGL((dropout_kernel<kBF16>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dropout_kernel<kF16>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace maxsim
