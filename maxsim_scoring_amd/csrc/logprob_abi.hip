// The C ABI declared in include/maxsim_loss.h: host-side validation (before
// anything is enqueued), then one launcher per entry point.
#include "maxsim_loss.h"

#include <climits>

#include "logprob.hpp"

using namespace maxsim;

namespace {

constexpr int64_t kMax = ((int64_t)1 << 31) - kLpChunk;  // the end of a row's last chunk stays below 2^31
constexpr int64_t kI32Max = INT32_MAX;

maxsim_status_t launch_status(hipError_t e) { return e == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH; }

bool float_ok(maxsim_dtype_t t) { return t == MAXSIM_F16 || t == MAXSIM_BF16 || t == MAXSIM_F32; }
int elem_of(maxsim_dtype_t t) { return t == MAXSIM_F16 ? kF16 : t == MAXSIM_BF16 ? kBF16 : kF32; }
uintptr_t bytes_of(maxsim_dtype_t t) { return t == MAXSIM_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// Where a difference of scores overflows, its probability is 0; NaN is not in it.
bool scale_ok(float s) { return s >= 0x1p-64f && s <= 0x1p64f; }

int64_t chunks_of(int64_t Nd) { return Nd > kLpChunk ? (Nd + kLpChunk - 1) / kLpChunk : 1; }

// Sizes that neither an index nor a grid overflows with; Nq > 0.
bool sizes_ok(int64_t Nq, int64_t Nd, int64_t P)
{
    if (Nq >= kMax || Nd >= kMax || P >= kMax) return false;
    return Nq * chunks_of(Nd) <= kI32Max && (P == 0 || Nq <= kI32Max / P);
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

// Byte offsets of the workspace's parts, and its size.
struct Parts {
    int64_t cand, top, rank, size;
    Parts(int64_t Nq, int64_t Nd, int64_t P, int64_t K)
    {
        const int64_t u = Nq * chunks_of(Nd);
        cand = u * 16;
        top = align16(cand + u * 8 * logprob_cap(K));
        rank = align16(top + u * 4);
        size = align16(rank + u * 4 * P);
    }
};

void columns(LogprobArgs& a, int64_t Nd)
{
    a.Nd = (int32_t)Nd;
    a.chunks = (int32_t)chunks_of(Nd);
    a.cbits = 1;
    while (a.cbits < 31 && ((int64_t)1 << a.cbits) < Nd) ++a.cbits;
}

}  // namespace

extern "C" {

int64_t maxsim_logprob_workspace(int64_t Nq, int64_t Nd, int64_t P, int64_t K)
{
    if (Nq < 0 || Nd < 0 || P < 0 || K < 0 || K > MAXSIM_LOGPROB_MAX_K) return -1;
    if (Nq == 0) return 0;
    if (!sizes_ok(Nq, Nd, P)) return -1;
    return chunks_of(Nd) == 1 ? 0 : Parts(Nq, Nd, P, K).size;
}

maxsim_status_t maxsim_logprob_fwd(maxsim_dtype_t dtype, const void* X, int64_t Nq, int64_t Nd,
                                   float scale, const uint8_t* mask, const int32_t* targets,
                                   int64_t P, int64_t K, float* logp, int32_t* rank, float* norm,
                                   float* entropy, int32_t* top_idx, float* top_logp,
                                   void* workspace, int64_t workspace_bytes,
                                   maxsim_stream_t stream)
{
    if (Nq < 0 || Nd < 0 || P < 0 || K < 0 || workspace_bytes < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || K > MAXSIM_LOGPROB_MAX_K || !scale_ok(scale)) return MAXSIM_ERR_UNSUPPORTED;
    if (Nq == 0) return MAXSIM_OK;
    if ((Nd > 0 && !X) || (P > 0 && (!targets || !logp)) || !norm || (K > 0 && (!top_idx || !top_logp)))
        return MAXSIM_ERR_NULL;
    if (!aligned(X, bytes_of(dtype)) || !aligned(targets, 4) || !aligned(logp, 4) || !aligned(rank, 4) ||
        !aligned(norm, 4) || !aligned(entropy, 4) || !aligned(top_idx, 4) || !aligned(top_logp, 4) ||
        !aligned(workspace, 16))
        return MAXSIM_ERR_UNSUPPORTED;
    if (!sizes_ok(Nq, Nd, P)) return MAXSIM_ERR_OVERFLOW;
    LogprobArgs a{};
    columns(a, Nd);
    if (a.chunks > 1) {
        const Parts at(Nq, Nd, P, K);
        if (!workspace) return MAXSIM_ERR_NULL;
        if (workspace_bytes < at.size) return MAXSIM_ERR_SHAPE;
        char* w = (char*)workspace;
        a.ws_sums = (double*)w;
        a.ws_cand = (uint64_t*)(w + at.cand);
        a.ws_top = (float*)(w + at.top);
        a.ws_rank = (uint32_t*)(w + at.rank);
    }
    a.X = X;
    a.mask = mask;
    a.targets = targets;
    a.Nq = Nq;
    a.P = (int32_t)P;
    a.K = (int32_t)K;
    a.cap = logprob_cap(K);
    a.scale = scale;
    a.logp = logp;
    a.rank = P > 0 ? rank : nullptr;
    a.norm = norm;
    a.entropy = entropy;
    a.top_idx = top_idx;
    a.top_logp = top_logp;
    return launch_status(launch_logprob_fwd(elem_of(dtype), a, (hipStream_t)stream));
}

maxsim_status_t maxsim_logprob_bwd(maxsim_dtype_t dtype, const void* X, int64_t Nq, int64_t Nd,
                                   float scale, const uint8_t* mask, const int32_t* targets,
                                   int64_t P, const float* norm, const float* entropy,
                                   const float* grad_logp, const float* grad_entropy,
                                   maxsim_dtype_t dx_dtype, void* dX, maxsim_stream_t stream)
{
    if (Nq < 0 || Nd < 0 || P < 0) return MAXSIM_ERR_SHAPE;
    if (!float_ok(dtype) || !float_ok(dx_dtype) || !scale_ok(scale)) return MAXSIM_ERR_UNSUPPORTED;
    if (Nq == 0 || Nd == 0) return MAXSIM_OK;
    if (!X || !norm || !dX || (P > 0 && (!targets || !grad_logp)) || !entropy != !grad_entropy) return MAXSIM_ERR_NULL;
    if (!aligned(X, bytes_of(dtype)) || !aligned(targets, 4) || !aligned(norm, 4) || !aligned(entropy, 4) ||
        !aligned(grad_logp, 4) || !aligned(grad_entropy, 4) || !aligned(dX, bytes_of(dx_dtype)))
        return MAXSIM_ERR_UNSUPPORTED;
    if (!sizes_ok(Nq, Nd, P)) return MAXSIM_ERR_OVERFLOW;
    LogprobArgs a{};
    columns(a, Nd);
    a.X = X;
    a.mask = mask;
    a.targets = targets;
    a.Nq = Nq;
    a.P = (int32_t)P;
    a.scale = scale;
    a.norm_in = norm;
    a.entropy_in = entropy;
    a.g_logp = grad_logp;
    a.g_entropy = grad_entropy;
    a.dX = dX;
    a.out = elem_of(dx_dtype);
    return launch_status(launch_logprob_bwd(elem_of(dtype), a, (hipStream_t)stream));
}

}  // extern "C"
