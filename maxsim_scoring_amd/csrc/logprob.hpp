// Log probabilities of given columns of score rows: argument blocks, launchers.
#pragma once

#include "embed_common.hpp"

namespace maxsim {

constexpr int kLpValues = 16;                     // columns a thread holds
constexpr int kLpChunk = 256 * kLpValues;         // columns of a workgroup

struct LogprobArgs {
    const void* X;           // [Nq, Nd]
    const uint8_t* mask;     // [Nq, Nd] or null
    const int32_t* targets;  // [Nq, P]
    int64_t Nq;
    int32_t Nd, P, K;
    float scale;
    // forward
    float* logp;        // [Nq, P]
    int32_t* rank;      // [Nq, P] or null
    float* norm;        // [Nq, 2]
    float* entropy;     // [Nq] or null
    int32_t* top_idx;   // [Nq, K]
    float* top_logp;    // [Nq, K]
    // workspace of rows of several chunks: of each (row, chunk)
    double* ws_sums;    // sum of 2^t, sum of 2^t t; t against the chunk's largest
    uint64_t* ws_cand;  // [cap] candidates for the best columns, 0 behind the last
    float* ws_top;      // the largest score
    uint32_t* ws_rank;  // [P] candidates before each target
    int32_t chunks;     // of a row
    int32_t cap;        // most candidates that one selection may leave
    int32_t cbits;      // bits of a column
    // backward
    const float* norm_in;
    const float* entropy_in;
    const float* g_logp;
    const float* g_entropy;
    void* dX;
    int out;  // element type of dX
};

// The most candidates that a selection of K leaves: some more than K, so that it
// seldom has to tell the last few apart.
inline int logprob_cap(int64_t K) { return K == 0 ? 0 : (int)(K + K / 2 + 32); }

hipError_t launch_logprob_fwd(int elem, LogprobArgs a, hipStream_t stream);
hipError_t launch_logprob_bwd(int elem, LogprobArgs a, hipStream_t stream);

}  // namespace maxsim
