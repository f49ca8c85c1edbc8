// The C ABI declared in include/maxsim_mx4.h: host-side validation (before
// anything is enqueued), then one launcher per entry point.
#include "maxsim_mx4.h"

#include <climits>

#include "mx4_common.hpp"

using namespace maxsim;

namespace {

constexpr int64_t kI32Max = INT32_MAX;
constexpr int64_t kMaxChannels = (int64_t)1 << 26;  // 2^22 workgroups of 16 channels

maxsim_status_t launch_status(hipError_t e) { return e == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH; }

bool float_ok(maxsim_dtype_t t) { return t == MAXSIM_F16 || t == MAXSIM_BF16 || t == MAXSIM_F32; }
int elem_of(maxsim_dtype_t t) { return t == MAXSIM_F16 ? kF16 : t == MAXSIM_BF16 ? kBF16 : kF32; }
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool width_ok(int64_t d) { return d >= 1 && d <= MAXSIM_MX4_MAX_WIDTH; }
int32_t blocks(int64_t d) { return (int32_t)((d + 31) / 32); }

// The checks that both directions of the conversion share; *done is set when
// there is nothing left to do (an error, or no rows).
maxsim_status_t check_rows(maxsim_dtype_t dtype, const void* X, int64_t T, int64_t d, const void* codes,
                           const void* scale, bool* done)
{
    *done = true;
    if (T < 0 || d < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || !width_ok(d)) return MAXSIM_ERR_UNSUPPORTED;
    if (T == 0) return MAXSIM_OK;
    if (!X || !codes || !scale) return MAXSIM_ERR_NULL;
    if (!aligned(X, 16) || !aligned(codes, 16)) return MAXSIM_ERR_UNSUPPORTED;
    if (T > kI32Max) return MAXSIM_ERR_OVERFLOW;
    *done = false;
    return MAXSIM_OK;
}

}  // namespace

extern "C" {

maxsim_status_t maxsim_quantize_mx4(maxsim_dtype_t dtype, const void* X, int64_t T, int64_t d,
                                    const uint8_t* mask, int normalize, uint8_t* codes,
                                    uint8_t* scale, maxsim_stream_t stream)
{
    bool done;
    const maxsim_status_t st = check_rows(dtype, X, T, d, codes, scale, &done);
    if (done) return st;
    Mx4RowArgs a{};
    a.X = X;
    a.mask = mask;
    a.codes = codes;
    a.scale = scale;
    a.T = T;
    a.d = (int32_t)d;
    a.nb = blocks(d);
    return launch_status(launch_quantize_mx4(elem_of(dtype), a, normalize != 0, (hipStream_t)stream));
}

maxsim_status_t maxsim_dequantize_mx4(const uint8_t* codes, const uint8_t* scale, int64_t T,
                                      int64_t d, maxsim_dtype_t dtype, void* Y,
                                      maxsim_stream_t stream)
{
    bool done;
    const maxsim_status_t st = check_rows(dtype, Y, T, d, codes, scale, &done);
    if (done) return st;
    Mx4RowArgs a{};
    a.codes = const_cast<uint8_t*>(codes);
    a.scale = const_cast<uint8_t*>(scale);
    a.Y = Y;
    a.T = T;
    a.d = (int32_t)d;
    a.nb = blocks(d);
    a.out = elem_of(dtype);
    return launch_status(launch_dequantize_mx4(a, (hipStream_t)stream));
}

maxsim_status_t maxsim_linear_mx4(maxsim_dtype_t dtype, const uint8_t* A, const uint8_t* a_scale,
                                  const uint8_t* W, const uint8_t* w_scale, const float* bias,
                                  int64_t T, int64_t N, int64_t K, void* Y,
                                  maxsim_stream_t stream)
{
    if (T < 0 || N < 0 || K < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || !width_ok(K) || N < 1) return MAXSIM_ERR_UNSUPPORTED;
    if (T == 0) return MAXSIM_OK;
    if (!A || !a_scale || !W || !w_scale || !Y) return MAXSIM_ERR_NULL;
    if (!aligned(A, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(bias, 4)) return MAXSIM_ERR_UNSUPPORTED;
    if (T > kI32Max || N > kMaxChannels) return MAXSIM_ERR_OVERFLOW;
    Mx4LinearArgs a{};
    a.A = A;
    a.a_scale = a_scale;
    a.W = W;
    a.w_scale = w_scale;
    a.bias = bias;
    a.Y = Y;
    a.T = T;
    a.N = (int32_t)N;
    a.nb = blocks(K);
    a.out = elem_of(dtype);
    return launch_status(launch_linear_mx4(a, (hipStream_t)stream));
}

maxsim_status_t maxsim_fwd_mx4(const uint8_t* Q, const uint8_t* q_scale, const uint8_t* D,
                               const uint8_t* d_scale, int64_t Nq, int64_t Nd, int64_t Lq,
                               int64_t Ld, int64_t d, const uint8_t* q_mask,
                               const uint8_t* d_mask, float* scores, int32_t* argmax,
                               maxsim_stream_t stream)
{
    if (Nq < 0 || Nd < 0 || Lq < 0 || Ld < 0 || d < 0) return MAXSIM_ERR_SHAPE;
    if (d < 1 || d > 1024) return MAXSIM_ERR_UNSUPPORTED;
    if (Nq == 0 || Nd == 0) return MAXSIM_OK;
    if (!scores || (Lq > 0 && (!Q || !q_scale)) || (Ld > 0 && (!D || !d_scale))) return MAXSIM_ERR_NULL;
    if (!aligned(Q, 16) || !aligned(D, 16) || !aligned(scores, 4) || !aligned(argmax, 4)) return MAXSIM_ERR_UNSUPPORTED;
    if (Nq > kI32Max - 64 || Lq > kI32Max - 64 || Ld > kI32Max - 64 || Nd > kI32Max) return MAXSIM_ERR_OVERFLOW;
    if (Nq * Nd > kI32Max || (argmax && Lq > 0 && Nq * Nd > kI32Max / Lq)) return MAXSIM_ERR_OVERFLOW;
    Mx4FwdArgs a{};
    a.Q = Q;
    a.q_scale = q_scale;
    a.D = D;
    a.d_scale = d_scale;
    a.q_mask = q_mask;
    a.d_mask = d_mask;
    a.scores = scores;
    a.argmax = argmax;
    a.Nq = Nq;
    a.Nd = Nd;
    a.Lq = Lq;
    a.Ld = Ld;
    a.nb = blocks(d);
    return launch_status(launch_fwd_mx4(a, (hipStream_t)stream));
}

}  // extern "C"
