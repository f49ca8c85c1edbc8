// Cross-product MaxSim of microscaled 4-bit queries and documents: the kernels of several
// queries of up to 16 tokens, which share tiles.
#include "fwd_mx4.hpp"

namespace maxsim {

namespace {

template <int G, int NTW, int P, int WAVES>
void run_packed(Mx4FwdArgs a, hipStream_t stream)
{
    a.qpw = NTW * (32 >> a.log2_qslot);
    a.nqb = (int32_t)pieces(a.Nq, a.qpw);
    const int64_t units = (int64_t)device_cu_count() * WAVES, want = units / a.nqb > 0 ? units / a.nqb : 1;
    a.nranges = (int32_t)(want < a.Nd ? want : a.Nd);
    const dim3 grid((unsigned)pieces((int64_t)a.nqb * a.nranges, kWaves)), block(kWaves * 64);
    const bool fast = fast_rows<G>(a);
    // (more query registers beside an argmax's would spill)
    if constexpr (NTW == 1 || G == 1) {
        if (a.argmax && fast) hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, true, true, kPacked>), grid, block, 0, stream, a);
        else if (a.argmax) hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, true, false, kPacked>), grid, block, 0, stream, a);
    }
    if (!a.argmax && fast) hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, false, true, kPacked>), grid, block, 0, stream, a);
    else if (!a.argmax) hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, false, false, kPacked>), grid, block, 0, stream, a);
}

}  // namespace

// 64 queries of one token over 20,000 documents of 100 tokens take 31 us, 362 with a tile
// for each query; 32 of 5 over 5000 of 180 24 and 64; 6 of 16 over 17,302 of 90 28 and
// 44. Tiles a wave as for longer queries. False where no tile would be shared.
bool launch_fwd_mx4_packed(Mx4FwdArgs a, hipStream_t stream)
{
    if (a.Lq > 16 || a.Nq < 2) return false;
    a.log2_qslot = log2_up(a.Lq);
    const int64_t tiles = pieces(a.Nq, 32 >> a.log2_qslot);
    const bool many = tiles > 1 && tiles * a.Nd >= 16 * (int64_t)device_cu_count() && (!a.argmax || a.nb <= 4);
    if (a.nb <= 4) {
        if (many) run_packed<1, 4, 2, 12>(a, stream);
        else run_packed<1, 1, 4, 16>(a, stream);
    } else if (a.nb <= 8) {
        if (many) run_packed<2, 4, 2, 8>(a, stream);
        else run_packed<2, 1, 3, 8>(a, stream);
    } else if (a.nb <= 12) {
        if (many) run_packed<3, 4, 2, 8>(a, stream);
        else run_packed<3, 1, 2, 12>(a, stream);
    } else if (a.nb <= 16) {
        if (many) run_packed<4, 4, 2, 8>(a, stream);
        else run_packed<4, 1, 2, 8>(a, stream);
    } else if (a.nb <= 24) {
        if (many) run_packed<6, 4, 2, 4>(a, stream);
        else run_packed<6, 1, 2, 8>(a, stream);
    } else {
        if (many) run_packed<8, 2, 2, 4>(a, stream);
        else run_packed<8, 1, 2, 4>(a, stream);
    }
    return true;
}

}  // namespace maxsim
