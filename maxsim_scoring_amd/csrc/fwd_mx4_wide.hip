// Cross-product MaxSim of microscaled 4-bit queries and documents: the kernels of more
// than 256 channels.
#include "fwd_mx4.hpp"

namespace maxsim {

// n: query tiles a wave that leave work for all. A width between the classes takes the
// kernel above it: one query over 10,000 documents of 180 tokens 51.9 us at 384 channels,
// 80 at 512, 138 at 640, 123 at 768, 268 at 896 and 149 at 1024 (exponents of whole words
// only where all of a class's blocks are there).
void launch_fwd_mx4_wide(const Mx4FwdArgs& a, int n, hipStream_t stream)
{
    if (a.nb <= 12) {
        if (n >= 3) run<3, 4, 2, 8>(a, stream);
        else run<3, 1, 2, 12>(a, stream);
    } else if (a.nb <= 16) {
        if (n >= 3 && !a.argmax) run<4, 4, 2, 8>(a, stream);
        else if (n >= 2) run<4, 2, 2, 8>(a, stream);
        else run<4, 1, 2, 8, true>(a, stream);
    } else if (a.nb <= 24) {
        if (n >= 3 && !a.argmax) run<6, 4, 2, 4>(a, stream);
        else if (n >= 2) run<6, 2, 2, 4>(a, stream);
        else run<6, 1, 2, 8, true>(a, stream);
    } else {
        if (n >= 2) run<8, 2, 2, 4>(a, stream);
        else run<8, 1, 2, 4, true>(a, stream);
    }
}

}  // namespace maxsim
