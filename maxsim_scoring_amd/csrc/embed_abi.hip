// The C ABI declared in include/maxsim_embed.h: host-side validation (before
// anything is enqueued), then one launcher per entry point.
#include "maxsim_embed.h"

#include <climits>
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"

using namespace maxsim;

namespace {

constexpr int64_t kI32Max = INT32_MAX;
constexpr int64_t kMaxChannels = (int64_t)1 << 26;  // 2^22 workgroups of 16 channels
constexpr int64_t kMaxElems = (int64_t)1 << 43;  // dropout: keeps every index product in 64 bits

maxsim_status_t launch_status(hipError_t e) { return e == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH; }

bool float_ok(maxsim_dtype_t t) { return t == MAXSIM_F16 || t == MAXSIM_BF16 || t == MAXSIM_F32; }

int elem_of(maxsim_dtype_t t)
{
    return t == MAXSIM_F16 ? kF16 : t == MAXSIM_BF16 ? kBF16 : t == MAXSIM_I8 ? kI8 : kF32;
}

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool width_ok(int64_t d) { return d >= 1 && d <= MAXSIM_EMBED_MAX_WIDTH; }

maxsim_status_t dropout(maxsim_dtype_t dtype, const void* X, int64_t n, double p, uint64_t seed,
                        uint64_t step, const uint64_t* step_dev, void* Y, maxsim_stream_t stream)
{
    if (n < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || !(p >= 0.0 && p <= 1.0)) return MAXSIM_ERR_UNSUPPORTED;  // NaN p too
    if (n == 0) return MAXSIM_OK;
    if (!X || !Y) return MAXSIM_ERR_NULL;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(step_dev, 8)) return MAXSIM_ERR_UNSUPPORTED;
    if (n >= kMaxElems) return MAXSIM_ERR_OVERFLOW;
    DropArgs a{};
    a.X = X;
    a.Y = Y;
    a.n = n;
    a.seed_lo = (uint32_t)seed;
    a.seed_hi = (uint32_t)(seed >> 32);
    a.step = step;
    a.step_dev = step_dev;
    a.q = (uint32_t)std::floor(p * 65536.0 + 0.5);
    a.up = a.q < 65536 ? (float)(65536.0 / (65536.0 - a.q)) : 0.0f;
    return launch_status(launch_dropout(elem_of(dtype), a, (hipStream_t)stream));
}

// The checks that maxsim_linear_i8 and maxsim_embed_i8 share; *done is set
// when there is nothing left to do (an error, or no rows).
maxsim_status_t check_linear(const int8_t* A, const float* a_scale, const int8_t* W,
                             const float* w_scale, const float* bias, int64_t T, int64_t N,
                             int64_t K, const void* Y, bool* done)
{
    *done = true;
    if (T == 0) return MAXSIM_OK;
    if (!A || !a_scale || !W || !w_scale || !Y) return MAXSIM_ERR_NULL;
    if (!aligned(A, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(a_scale, 4) ||
        !aligned(w_scale, 4) || !aligned(bias, 4))
        return MAXSIM_ERR_UNSUPPORTED;
    if (T > kI32Max || N > kMaxChannels) return MAXSIM_ERR_OVERFLOW;
    *done = false;
    return MAXSIM_OK;
}

}  // namespace

extern "C" {

maxsim_status_t maxsim_quantize_tok(maxsim_dtype_t dtype, const void* X, int64_t T, int64_t d,
                                    const uint8_t* mask, int normalize, int8_t* codes,
                                    float* scale, maxsim_stream_t stream)
{
    if (T < 0 || d < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || !width_ok(d)) return MAXSIM_ERR_UNSUPPORTED;
    if (T == 0) return MAXSIM_OK;
    if (!X || !codes || !scale) return MAXSIM_ERR_NULL;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return MAXSIM_ERR_UNSUPPORTED;
    if (T > kI32Max) return MAXSIM_ERR_OVERFLOW;
    RowArgs a{};
    a.X = X;
    a.mask = mask;
    a.Y = codes;
    a.stat = scale;
    a.T = T;
    a.d = (int32_t)d;
    a.normalize = normalize != 0;
    return launch_status(launch_quantize(elem_of(dtype), a, (hipStream_t)stream));
}

maxsim_status_t maxsim_normalize_fwd(maxsim_dtype_t x_dtype, const void* X, int64_t T, int64_t d,
                                     const uint8_t* mask, maxsim_dtype_t y_dtype, void* Y,
                                     float* rnorm, maxsim_stream_t stream)
{
    if (T < 0 || d < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(x_dtype) || !float_ok(y_dtype) || !width_ok(d)) return MAXSIM_ERR_UNSUPPORTED;
    if (T == 0) return MAXSIM_OK;
    if (!X || !Y || !rnorm) return MAXSIM_ERR_NULL;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(rnorm, 4)) return MAXSIM_ERR_UNSUPPORTED;
    if (T > kI32Max) return MAXSIM_ERR_OVERFLOW;
    RowArgs a{};
    a.X = X;
    a.mask = mask;
    a.Y = Y;
    a.stat = rnorm;
    a.T = T;
    a.d = (int32_t)d;
    a.out = elem_of(y_dtype);
    return launch_status(launch_normalize_fwd(elem_of(x_dtype), a, (hipStream_t)stream));
}

maxsim_status_t maxsim_normalize_bwd(maxsim_dtype_t x_dtype, const void* X, const float* rnorm,
                                     const float* dY, int64_t T, int64_t d,
                                     maxsim_dtype_t dx_dtype, void* dX, maxsim_stream_t stream)
{
    if (T < 0 || d < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(x_dtype) || !float_ok(dx_dtype) || !width_ok(d)) return MAXSIM_ERR_UNSUPPORTED;
    if (T == 0) return MAXSIM_OK;
    if (!X || !rnorm || !dY || !dX) return MAXSIM_ERR_NULL;
    if (!aligned(X, 16) || !aligned(dY, 16) || !aligned(dX, 16) || !aligned(rnorm, 4))
        return MAXSIM_ERR_UNSUPPORTED;
    if (T > kI32Max) return MAXSIM_ERR_OVERFLOW;
    RowArgs a{};
    a.X = X;
    a.rnorm = rnorm;
    a.g = dY;
    a.Y = dX;
    a.T = T;
    a.d = (int32_t)d;
    a.out = elem_of(dx_dtype);
    return launch_status(launch_normalize_bwd(elem_of(x_dtype), a, (hipStream_t)stream));
}

maxsim_status_t maxsim_dropout_fwd(maxsim_dtype_t dtype, const void* X, int64_t n, double p,
                                   uint64_t seed, uint64_t step, const uint64_t* step_dev, void* Y,
                                   maxsim_stream_t stream)
{
    return dropout(dtype, X, n, p, seed, step, step_dev, Y, stream);
}

maxsim_status_t maxsim_dropout_bwd(maxsim_dtype_t dtype, const void* dY, int64_t n, double p,
                                   uint64_t seed, uint64_t step, const uint64_t* step_dev, void* dX,
                                   maxsim_stream_t stream)
{
    return dropout(dtype, dY, n, p, seed, step, step_dev, dX, stream);
}

maxsim_status_t maxsim_linear_i8(maxsim_dtype_t dtype, const int8_t* A, const float* a_scale,
                                 const int8_t* W, const float* w_scale, const float* bias,
                                 int64_t T, int64_t N, int64_t K, void* Y,
                                 maxsim_stream_t stream)
{
    if (T < 0 || N < 0 || K < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || !width_ok(K) || N < 1) return MAXSIM_ERR_UNSUPPORTED;
    bool done;
    const maxsim_status_t st = check_linear(A, a_scale, W, w_scale, bias, T, N, K, Y, &done);
    if (done) return st;
    LinearArgs a{};
    a.A = A;
    a.a_scale = a_scale;
    a.W = W;
    a.w_scale = w_scale;
    a.bias = bias;
    a.Y = Y;
    a.T = T;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.out = elem_of(dtype);
    return launch_status(launch_linear_i8(a, (hipStream_t)stream));
}

maxsim_status_t maxsim_embed_i8(maxsim_dtype_t dtype, const int8_t* A, const float* a_scale,
                                const int8_t* W, const float* w_scale, const float* bias,
                                const uint8_t* mask, int64_t T, int64_t d, int64_t K, void* E,
                                float* e_scale, maxsim_stream_t stream)
{
    if (T < 0 || d < 0 || K < 0) return MAXSIM_ERR_SHAPE;
    if (!(float_ok(dtype) || dtype == MAXSIM_I8) || !width_ok(K) || d < 1 || d > MAXSIM_EMBED_MAX_DIM)
        return MAXSIM_ERR_UNSUPPORTED;
    bool done;
    const maxsim_status_t st = check_linear(A, a_scale, W, w_scale, bias, T, d, K, E, &done);
    if (done) return st;
    if (dtype == MAXSIM_I8 && !e_scale) return MAXSIM_ERR_NULL;
    if (!aligned(e_scale, 4)) return MAXSIM_ERR_UNSUPPORTED;
    LinearArgs a{};
    a.A = A;
    a.a_scale = a_scale;
    a.W = W;
    a.w_scale = w_scale;
    a.bias = bias;
    a.mask = mask;
    a.Y = E;
    a.y_scale = e_scale;
    a.T = T;
    a.N = (int32_t)d;
    a.K = (int32_t)K;
    a.out = elem_of(dtype);
    return launch_status(launch_embed_i8(a, (hipStream_t)stream));
}

}  // extern "C"
