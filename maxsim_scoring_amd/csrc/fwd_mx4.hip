// Cross-product MaxSim of microscaled 4-bit queries and documents: the dispatch, and
// the kernels of up to 256 channels.
#include "fwd_mx4.hpp"

namespace maxsim {

namespace {

// Scores (and argmax) where queries or documents have no tokens.
__global__ __launch_bounds__(256) void zero_mx4_kernel(Mx4FwdArgs a)
{
    const int64_t n = a.Nq * a.Nd, at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t k = at; k < n; k += step) a.scores[k] = 0.0f;
    if (a.argmax)
        for (int64_t k = at; k < n * a.Lq; k += step) a.argmax[k] = 0;
}

// Query tiles a wave: as many as leave work for all (n). Where the matrix cores are
// the bound 8 are ahead (32 queries of 32 over 1000 pages of 1024 tokens 66 us, 128 of
// 128 over 128 pages 108); 4 queries over 50,000 documents of 180 take 109 us with 4 a
// wave and 16 waves on a CU, 138 with 8 waves, one query 95 with 20 waves and 100
// with 8.
void scores_once(Mx4FwdArgs a, hipStream_t stream)
{
    if (launch_fwd_mx4_short(a, stream) || launch_fwd_mx4_packed(a, stream)) return;
    const int64_t tiles = a.Nq * a.ntq;
    const int64_t most = tiles * a.Nd / ((int64_t)device_cu_count() * 8);
    int n = (int)(most < tiles ? (most > 1 ? most : 1) : tiles);
    // a query of a few tiles stays in one wave, a longer one in one pass of four
    const int least = a.ntq <= 4 ? a.ntq : (a.ntq + 3) / 4;
    n = n > least ? n : least;
    if (a.nb > 8) {
        launch_fwd_mx4_wide(a, n, stream);
    } else if (a.nb <= 4) {
        if (n >= 8 && !a.argmax) run<1, 8, 2, 8>(a, stream);
        else if (n >= 3) run<1, 4, 2, 16>(a, stream);
        else if (n == 2) run<1, 2, 4, 12>(a, stream);
        else run<1, 1, 4, 20, true>(a, stream);
    } else {
        if (n >= 3) run<2, 4, 2, 8>(a, stream);
        else run<2, 1, 3, 8>(a, stream);
    }
}

}  // namespace

hipError_t launch_fwd_mx4(Mx4FwdArgs a, hipStream_t stream)
{
    if (a.Lq == 0 || a.Ld == 0) {
        const int64_t b = pieces(a.Nq * a.Nd * (a.argmax && a.Lq > 1 ? a.Lq : 1), 256);
        hipLaunchKernelGGL(zero_mx4_kernel, dim3((unsigned)(b < 65536 ? b : 65536)), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    a.ntq = (int32_t)pieces(a.Lq, 32);
    // One launch covers at most `step` queries, so that a grid's threads stay below
    // 2^32 (a query takes a workgroup at most); queries are independent.
    const int64_t step = (int64_t)1 << 20;
    for (int64_t left = a.Nq; left > 0; left -= step) {
        a.Nq = left < step ? left : step;
        scores_once(a, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.Q += step * a.Lq * a.nb * 16;
        a.q_scale += step * a.Lq * a.nb;
        if (a.q_mask) a.q_mask += step * a.Lq;
        a.scores += step * a.Nd;
        if (a.argmax) a.argmax += step * a.Nd * a.Lq;
    }
    return hipSuccess;
}

}  // namespace maxsim
