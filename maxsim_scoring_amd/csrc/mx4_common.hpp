// Microscaled 4-bit rows: argument blocks, launchers and device helpers.
#pragma once

#include "embed_common.hpp"

namespace maxsim {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Rows to codes and back.
struct Mx4RowArgs {
    const void* X;         // [T, d] (codes of the way back: null)
    const uint8_t* mask;   // [T] or null
    uint8_t* codes;        // [T, 16 nb]
    uint8_t* scale;        // [T, nb]
    void* Y;               // [T, d] (the way back)
    int64_t T;
    int32_t d, nb;
    int32_t log2_lanes;    // lanes that share a row
    int out;               // element type of Y
};

struct Mx4LinearArgs {
    const uint8_t* A;        // [T, 16 nb]
    const uint8_t* a_scale;  // [T, nb]
    const uint8_t* W;        // [N, 16 nb]
    const uint8_t* w_scale;  // [N, nb]
    const float* bias;       // [N] or null
    void* Y;                 // [T, N]
    int64_t T;
    int32_t N, nb;
    int out;
    // filled by the launcher
    int32_t tiles_t, tiles_n;
};

struct Mx4FwdArgs {
    const uint8_t* Q;        // [Nq, Lq, 16 nb]
    const uint8_t* q_scale;  // [Nq, Lq, nb]
    const uint8_t* D;        // [Nd, Ld, 16 nb]
    const uint8_t* d_scale;  // [Nd, Ld, nb]
    const uint8_t* q_mask;   // [Nq, Lq] or null
    const uint8_t* d_mask;   // [Nd, Ld] or null
    float* scores;           // [Nq, Nd]
    int32_t* argmax;         // [Nq, Nd, Lq] or null
    int64_t Nq, Nd, Lq, Ld;
    int32_t nb;
    // filled by the launcher
    int32_t ntq;      // 32-token tiles of a query
    int32_t qpw;      // whole queries of a unit
    int32_t nqb;      // blocks of queries
    int32_t nranges;  // ranges of documents
    int32_t log2_slot, log2_qslot;  // rows of a short document, columns of a query (5: of a tile)
};

hipError_t launch_quantize_mx4(int elem, Mx4RowArgs a, bool normalize, hipStream_t stream);
hipError_t launch_dequantize_mx4(Mx4RowArgs a, hipStream_t stream);
hipError_t launch_linear_mx4(Mx4LinearArgs a, hipStream_t stream);
hipError_t launch_fwd_mx4(Mx4FwdArgs a, hipStream_t stream);
void launch_fwd_mx4_wide(const Mx4FwdArgs& a, int n, hipStream_t stream);
bool launch_fwd_mx4_short(Mx4FwdArgs a, hipStream_t stream);
bool launch_fwd_mx4_packed(Mx4FwdArgs a, hipStream_t stream);

// The block-scaled matrix product of 4-bit operands. A lane's 16 bytes are 32
// codes, one block: lane l of the 32-row form holds row l % 32, block l / 32 of
// two; of the 16-row form row l % 16, block l / 16 of four. Byte SA (SB) of its
// scale word is the block's exponent. (The intrinsic takes operands of up to 8
// bits; with format 4 the upper registers are not read.) The scales are taken from the
// lanes that EXEC enables, so all lanes have to get here. The compiler does not know
// that: a result that only some lanes use it computes in those lanes' branch, so one
// that may be used so is told to stay. (Sums that go round a loop cannot be moved out
// of it.)
__device__ __forceinline__ i32x8 widen(const i32x4& a) { return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1); }
template <int SA, int SB>
__device__ __forceinline__ f32x16 mfma32_mx4(const i32x4& a, int sa, const i32x4& b, int sb, const f32x16& c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, 4, 4, SA, sa, SB, sb);
}
// Behind the last of a result's products: it is there before the lanes part.
__device__ __forceinline__ void stay(f32x16& acc) { asm volatile("" : "+v"(acc)); }
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma16_mx4(const i32x4& a, int sa, const i32x4& b, int sb, const f32x4& c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, 4, 4, SA, sa, SB, sb);
}

}  // namespace maxsim
