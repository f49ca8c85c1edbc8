// 8-bit matrix product with a scale per token and per output channel, and the
// same product with every row normalised (and quantised), for gfx950.
//
//   y[t,n] = a_scale[t] w_scale[n] sum_k A[t,k] W[n,k] + bias[n]
//
// The product runs transposed on the int8 matrix cores, W . A^T: MFMA rows are
// output channels and columns are tokens, so a lane holds channels of one
// token. The statistics of a row (its norm and largest magnitude) are then
// sums and maxima inside a lane, over the lanes that share the token, and over
// the waves that split the channels.
//
// stream_kernel: embeddings of up to 256 channels, K up to 1024. The weights stay
// in registers and the hidden states pass once, so memory bounds it: 360,000 x 768
// states to 128 codes take 72 to 77 us (by card), 4.2 to 4.5 TB/s of states and
// codes, against 60 us for a copy of as many bytes.
// tile_kernel: BT tokens x BN channels per workgroup; A and W tiles of KB bytes
// along k stream through a ring in LDS by direct-to-LDS loads, with 16-byte
// chunks swizzled against bank conflicts. Large products are bound by the matrix
// cores and their power: 8192 x 4096 x 4096 in 118 to 125 us (by card), 2.2 to 2.3
// POP/s (an MFMA-only loop on such data reaches 3.4).
// few_kernel: a few tokens. W is the traffic; every fragment goes straight from
// memory to registers, waves split k, and LDS joins their sums. One token through
// 4096 x 4096 weights takes 5.3 us, 2.8 of them the launch. With join_kernel it
// also makes embeddings whose channels are spread over workgroups.
#include "embed_common.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(1)));  // at any address

// 16 bytes of a row of K bytes from byte k on (k a multiple of 16); bytes past
// the row's end are 0. UNAL: the row may start at any byte address. Only bytes
// of the row are read.
template <bool UNAL>
__device__ __forceinline__ i32x4 load16(const int8_t* row, int k, int K)
{
    if constexpr (!UNAL) {
        return k < K ? *(const i32x4*)(row + k) : i32x4{};
    } else {
        if (k + 16 <= K) {
            const i32x4_any v = *(const i32x4_any*)(row + k);
            return i32x4{v[0], v[1], v[2], v[3]};
        }
        if (k >= K) return i32x4{};
        if (K >= 16) {
            // the row's last 16 bytes, moved down by the bytes that lie before k
            const i32x4_any v = *(const i32x4_any*)(row + K - 16);
            unsigned __int128 x = (unsigned __int128)(((uint64_t)(uint32_t)v[3] << 32) | (uint32_t)v[2]) << 64 |
                                  (((uint64_t)(uint32_t)v[1] << 32) | (uint32_t)v[0]);
            x >>= 8 * (k + 16 - K);
            return i32x4{(int)(uint32_t)x, (int)(uint32_t)(x >> 32), (int)(uint32_t)(x >> 64), (int)(uint32_t)(x >> 96)};
        }
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (i < K) w[i / 4] |= (uint32_t)(uint8_t)row[i] << (8 * (i % 4));
        return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    }
}

// y in float32: the sum, the scales' product and the bias each round once (no
// fused multiply-add, so the result does not depend on the kernel).
__device__ __forceinline__ float scaled(int acc, float as, float ws, float b)
{
#pragma clang fp contract(off)
    const float s = as * ws;
    return (float)acc * s + b;
}
__device__ __forceinline__ double scaled64(int acc, double as, float ws, float b)
{
    return __builtin_fma((double)acc, as * (double)ws, (double)b);  // the scales' product is exact
}

// store_run for codes, four in a word.
template <int R>
__device__ __forceinline__ void store_codes(void* Y, int64_t t, int n, int N, const uint32_t (&w)[R / 4])
{
    int8_t* p = (int8_t*)Y + t * N + n;
    if ((N & 3) == 0) {
        if (R == 16 && (N & 15) == 0) {
            if (n < N) *(u32x4*)p = u32x4{w[0], w[R / 4 > 1 ? 1 : 0], w[R / 4 > 2 ? 2 : 0], w[R / 4 > 3 ? 3 : 0]};
        } else {
#pragma unroll
            for (int i = 0; i < R / 4; ++i)
                if (n + 4 * i < N) ((uint32_t*)p)[i] = w[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (n + i < N) p[i] = (int8_t)(w[i / 4] >> 8 * (i % 4));
}

__device__ __forceinline__ double xor_lane(double v, int m) { return __shfl_xor(v, m, 64); }

// The code of y in byte 2 of a word, inv about 127 / s: the fma adds 1/2 to
// 127 y / s, and 1.5 * 2^36, which leaves 16 bits of fraction in the low half.
// inv's rounding moves the sum by 2^-46 and the fma's by 2^-17, so the byte is the
// integer below the true sum unless those 16 bits are 0. Then (one value in 2^16,
// and every tie) tie_word decides.
__device__ __forceinline__ uint32_t code_word(double y, double inv, double magic)
{
    return (uint32_t)__builtin_bit_cast(uint64_t, __builtin_fma(y, inv, magic));
}
constexpr double kCodeMagic = 0x1.8p36 + 0.5;

// Byte 2 of `word`, m, or m - 1: which of them is nearest to 127 y / s, the even
// one on a tie. 254 y and (2 m - 1) s differ by less than 2^-15 of either, so their
// difference is exact in two parts: that of the rounded products, and that of
// what rounding took from them (both products have 61 bits).
__device__ __forceinline__ uint32_t tie_word(uint32_t word, double y, double s)
{
#pragma clang fp contract(off)
    const int m = (int)(word << 8) >> 24;
    const double c = (double)(2 * m - 1), p = 254.0 * y, q = c * s;
    const double over = (p - q) + (__builtin_fma(254.0, y, -p) - __builtin_fma(c, s, -q));
    const bool up = over > 0.0 || (over == 0.0 && (m & 1) == 0);
    return (uint32_t)(up ? m : m - 1) << 16;
}

// Four codes in a word.
__device__ __forceinline__ uint32_t pack_codes(const uint32_t (&q)[4])
{
    return __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0602u) | __builtin_amdgcn_perm(q[3], q[2], 0x0c0c0602u) << 16;
}

// The sums of one call, normalised and written in two halves with a barrier
// between them. For each of TT tokens a lane holds NB runs of R consecutive
// channels: sum(tt, b, i) is the int32 sum of channel chan(b) + i.
// ws and bs (LDS) hold the scales and biases of the workgroup's channels, 0 past
// the last one.
//
// With s the largest magnitude of the row, its values over the norm are
// (y / s) / ||y / s||, whose factors neither overflow nor vanish; the sum of
// squares is a float64, which holds the square of every float32 y. Codes are
// the nearest integers to 127 y / s, where y and s are float64: see code_word.
template <bool CODES, int TT, int NB, int R, int COLS, int WN>
struct Rows {
    // a lane's values stay in registers between the halves if they are few
    // (otherwise they are computed again: 64 to 128 of them would spill)
    static constexpr bool kKeep = TT * NB * R <= 16;
    double top[TT], ss[TT];
    double y64[CODES && kKeep ? 16 : 1];
    float y32[!CODES && kKeep ? 16 : 1];

    // Statistics of the lane's own channels.
    template <typename SUM, typename CHAN>
    __device__ __forceinline__ void first(SUM sum, CHAN chan, const float* ws, const float* bs, const float (&as)[TT],
                                          const bool (&live)[TT])
    {
        static_for<0, TT>([&](auto tt) {
            double m = 0.0, s2 = 0.0;
            float mf = 0.0f;
            static_for<0, NB>([&](auto b) {
                static_for<0, R>([&](auto i) {
                    const float w = ws[chan(b) + i], c = bs[chan(b) + i];
                    if constexpr (CODES) {
                        const double y = scaled64(sum(tt, b, i), (double)as[tt], w, c);
                        m = __builtin_fmax(m, __builtin_fabs(y));
                        s2 = __builtin_fma(y, y, s2);
                        if constexpr (kKeep) y64[(tt * NB + b) * R + i] = y;
                    } else {
                        const float y = scaled(sum(tt, b, i), as[tt], w, c);
                        mf = __builtin_fmaxf(mf, __builtin_fabsf(y));
                        s2 = __builtin_fma((double)y, (double)y, s2);
                        if constexpr (kKeep) y32[(tt * NB + b) * R + i] = y;
                    }
                });
                run_ends();
            });
            top[tt] = !live[tt] ? 0.0 : CODES ? m : (double)mf;
            ss[tt] = s2;
        });
    }

    // The sum again, as a value the compiler cannot tie to the first half's, and
    // the end of a run, over which it moves nothing: conversions kept or scales
    // loaded ahead for all runs would spill.
    static __device__ __forceinline__ int again(int s)
    {
        asm("" : "+v"(s));
        return s;
    }
    static __device__ __forceinline__ void run_ends()
    {
        if constexpr (!kKeep) __builtin_amdgcn_sched_barrier(0);
    }

    // Joins each token's statistics over the lanes that share it (lane / COLS), in a
    // fixed order, and leaves them for the WN waves that hold other channels in
    // red: 2 x WN rows of `stride`, slot the token's place. Waves that hold no
    // sums pass wn < 0.
    __device__ __forceinline__ void put(double* red, int stride, const int (&slot)[TT], int wn)
    {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int m = COLS; m < 64; m *= 2) {
                top[t] = __builtin_fmax(top[t], xor_lane(top[t], m));
                ss[t] += xor_lane(ss[t], m);
            }
        if (WN > 1 && wn >= 0 && lane_id() < COLS) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                red[wn * stride + slot[t]] = top[t];
                red[(WN + wn) * stride + slot[t]] = ss[t];
            }
        }
    }

    // After a barrier: the rows' statistics, and the outputs.
    template <typename SUM, typename CHAN>
    __device__ __forceinline__ void second(const LinearArgs& a, SUM sum, CHAN chan, const float* ws, const float* bs,
                                           const int64_t (&t)[TT], const float (&as)[TT], const bool (&live)[TT],
                                           const double* red, int stride, const int (&slot)[TT], int wn)
    {
        if constexpr (WN > 1) {
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                top[tt] = red[slot[tt]];
                ss[tt] = red[WN * stride + slot[tt]];
#pragma unroll
                for (int w = 1; w < WN; ++w) {
                    top[tt] = __builtin_fmax(top[tt], red[w * stride + slot[tt]]);
                    ss[tt] += red[(WN + w) * stride + slot[tt]];
                }
            }
        }
        // top leaves NaNs out, ss does not: a row with one is no zero row, and its
        // scale is NaN. Masked rows are zeros whatever the weights' scales and the
        // biases make of them.
        static_for<0, TT>([&](auto tt) {
            const bool in = t[tt] < a.T;
            const bool zero = !live[tt] || (top[tt] < (double)kTiny && !(ss[tt] != ss[tt]));
            if constexpr (!CODES) {
                const float inv = zero ? 0.0f : 1.0f / (float)top[tt];
                // the rest of the norm is between 1 and the square root of N
                const float r = zero ? 0.0f : rsqrt_f((float)(ss[tt] * (double)inv * (double)inv));
                static_for<0, NB>([&](auto b) {
                    float y[R];
                    static_for<0, R>([&](auto i) {
                        if constexpr (kKeep) y[i] = y32[(tt * NB + b) * R + i] * inv * r;
                        else y[i] = scaled(again(sum(tt, b, i)), as[tt], ws[chan(b) + i], bs[chan(b) + i]) * inv * r;
                    });
                    if (in) store_run<R>(a.Y, a.out, t[tt], chan(b), a.N, y, zero);
                    run_ends();
                });
            } else {
                const double inv = zero ? 0.0 : 127.0 / top[tt];
                double magic = kCodeMagic;
                asm("" : "+v"(magic));  // a register: as a constant it is copied for every fma
                static_for<0, NB>([&](auto b) {
                    auto value = [&](int i) {
                        if constexpr (kKeep) return y64[(tt * NB + b) * R + i];
                        else return scaled64(again(sum(tt, b, i)), (double)as[tt], ws[chan(b) + i], bs[chan(b) + i]);
                    };
                    constexpr int kPart = R / 4 < 2 ? R / 4 : 2;  // words decided together: more would spill
                    uint32_t w[R / 4];
                    static_for<0, R / 4 / kPart>([&](auto part) {
                        u16x2 least = {0xffff, 0xffff};  // the first: of the fractions
                        static_for<part * kPart, (part + 1) * kPart>([&](auto c) {
                            uint32_t q[4];
                            static_for<0, 4>([&](auto e) {
                                q[e] = code_word(value(c * 4 + e), inv, magic);
                                least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, q[e]));
                            });
                            w[c] = pack_codes(q);
                        });
                        if (__builtin_expect(least[0] == 0, 0)) {
                            double magic = kCodeMagic;  // formed again: words kept for this would spill too
                            asm("" : "+v"(magic));
                            static_for<part * kPart, (part + 1) * kPart>([&](auto c) {
                                uint32_t q[4];
                                static_for<0, 4>([&](auto e) {
                                    const double y = value(c * 4 + e);
                                    q[e] = code_word(y, inv, magic);
                                    if ((q[e] & 0xffffu) == 0) q[e] = tie_word(q[e], y, top[tt]);
                                    __builtin_amdgcn_sched_barrier(0);
                                });
                                w[c] = pack_codes(q);
                            });
                        }
                    });
                    static_for<0, R / 4>([&](auto c) { w[c] = zero ? 0 : w[c]; });
                    if (in) store_codes<R>(a.Y, t[tt], chan(b), a.N, w);
                    run_ends();
                });
                // codes * scale is y / ||y||, so scale = 1 / ||127 y / s||
                if (in && wn == 0 && lane_id() < COLS)
                    a.y_scale[t[tt]] = zero ? 1.0f : rsqrt_f((float)(ss[tt] * inv * inv));
            }
        });
    }
};

template <int TT, int NB, int R, int COLS, int WN, typename SUM, typename CHAN>
__device__ __forceinline__ void embed_rows(const LinearArgs& a, SUM sum, CHAN chan, const float* ws, const float* bs,
                                           const int64_t (&t)[TT], const float (&as)[TT], const bool (&live)[TT],
                                           const int (&slot)[TT], int wn, double* red, int stride)
{
    auto go = [&](auto& rows) {
        rows.first(sum, chan, ws, bs, as, live);
        rows.put(red, stride, slot, wn);
        if (WN > 1) block_barrier();
        rows.second(a, sum, chan, ws, bs, t, as, live, red, stride, slot, wn);
    };
    if (a.out == kI8) {
        Rows<true, TT, NB, R, COLS, WN> rows;
        go(rows);
    } else {
        Rows<false, TT, NB, R, COLS, WN> rows;
        go(rows);
    }
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------

template <int BT, int BN, int WT, int WN, int KB, int ST, bool EMBED, bool UNAL>
struct Tile {
    static constexpr int kWaves = WT * WN;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int TT = BT / WT / 32;  // 32-token column tiles per wave
    static constexpr int NT = BN / WN / 32;  // 32-channel row tiles per wave
    static constexpr int kCpr = KB / 16;     // chunks per row
    static constexpr int kLoads = (BT + BN) * kCpr / 64;              // wave-wide loads per stage
    static constexpr int kPerWave = (kLoads + kWaves - 1) / kWaves;
    static constexpr int kStage = (BT + BN) * KB;
    static constexpr int kRows = 64 / kCpr;  // rows of one load
    static_assert(BT % kRows == 0 && BN % kRows == 0, "a load stays inside one operand");
    static_assert(ST == 2 || kLoads % kWaves == 0, "deep rings count their loads");
    static_assert(EMBED || kWaves * 32 * (NT * 32 + 4) * 4 <= ST * kStage, "the ring holds a turned output");
};

// One stage's MFMAs: the wave's channels x tokens, KB bytes of k from `buf`.
template <typename C, int KB>
__device__ __forceinline__ void multiply(const uint8_t* buf, int w_row, int a_row, i32x16 (&acc)[C::NT][C::TT])
{
    const int l = lane_id() & 31, h = lane_id() >> 5;
#pragma unroll
    for (int ks = 0; ks < KB / 32; ++ks) {
        const int off = place<KB>(l, ks * 2 + h) * 16 + l * KB;
        i32x4 w[C::NT], x[C::TT];
#pragma unroll
        for (int i = 0; i < C::NT; ++i) w[i] = *(const i32x4*)(buf + (w_row + i * 32) * KB + off);
#pragma unroll
        for (int i = 0; i < C::TT; ++i) x[i] = *(const i32x4*)(buf + (a_row + i * 32) * KB + off);
#pragma unroll
        for (int i = 0; i < C::NT; ++i)
#pragma unroll
            for (int j = 0; j < C::TT; ++j) acc[i][j] = mfma32<kI8>(w[i], x[j], acc[i][j]);
    }
}

// Writes a wave's NT x 32 channels of TT x 32 tokens of a linear product, from
// channel n0 + wn * NT * 32 and token t0 + a_row on. ring: LDS of at least
// 32 x (NT * 32 + 4) floats per wave, free to overwrite.
template <int NT, int TT>
__device__ __forceinline__ void store_tile(const LinearArgs& a, const i32x16 (&acc)[NT][TT], const float* ws,
                                           const float* bs, int64_t t0, int n0, int a_row, int wn, int wave,
                                           uint8_t* ring)
{
    const int lane = lane_id(), half = lane >> 5;
    if (a.N & 3) {
        // Rows at any address: the wave turns its tokens x channels through LDS, so
        // that lanes store neighbouring channels (1213 x 1001 float32 outputs of
        // K = 1000: 11.9 us, 16.3 with every lane storing its own run value by value).
        constexpr int kCols = NT * 32, kStride = kCols + 4;
        float* mine = (float*)ring + wave * 32 * kStride;
        const int n_base = wn * kCols;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int64_t tile = t0 + a_row + j * 32, t = tile + (lane & 31);
            const float as = t < a.T ? a.a_scale[t] : 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int n = i * 32 + half * 16 + e;
                    mine[(lane & 31) * kStride + n] = scaled(acc[i][j][e], as, ws[n_base + n], bs[n_base + n]);
                }
            lds_fence();
            constexpr int kStep = kCols < 64 ? kCols : 64, kPer = 64 / kStep;  // columns and rows per store
            const int col = lane % kStep, sub = lane / kStep;
            for (int r = sub; r < 32 && tile + r < a.T; r += kPer) {
#pragma unroll
                for (int c = 0; c < kCols; c += kStep) {
                    const int n = n0 + n_base + c + col;
                    if (n >= a.N) continue;
                    const float y = mine[r * kStride + c + col];
                    const int64_t at = (tile + r) * a.N + n;
                    if (a.out == kF32) ((float*)a.Y)[at] = y;
                    else ((uint16_t*)a.Y)[at] = (uint16_t)half_bits(a.out, y);
                }
            }
            lds_fence();
        }
        return;
    }
    // 16-bit outputs whose channels all exist need no test per piece
    const bool whole = a.out != kF32 && (a.N & 7) == 0 && n0 + (wn + 1) * NT * 32 <= a.N;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = t0 + a_row + j * 32 + (lane & 31);
        if (t >= a.T) continue;
        const float as = a.a_scale[t];
        uint16_t* row = (uint16_t*)a.Y + t * a.N + n0;
        auto runs = [&](auto put) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int n = (wn * NT + i) * 32 + half * 16;
                float y[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = scaled(acc[i][j][e], as, ws[n + e], bs[n + e]);
                put(n, y);
            }
        };
        auto pack = [&](auto out) {
            runs([&](int n, const float (&y)[16]) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = half_pair<out>(y[2 * i], y[2 * i + 1]);
                ((u32x4*)(row + n))[0] = u32x4{w[0], w[1], w[2], w[3]};
                ((u32x4*)(row + n))[1] = u32x4{w[4], w[5], w[6], w[7]};
            });
        };
        if (whole && a.out == kBF16) pack(std::integral_constant<int, kBF16>{});
        else if (whole) pack(std::integral_constant<int, kF16>{});
        else runs([&](int n, const float (&y)[16]) { store_run<16>(a.Y, a.out, t, n0 + n, a.N, y); });
    }
}

// Workgroup to tile: consecutive workgroups go to the 8 XCDs in turn, so each XCD
// takes a contiguous run of tiles, walked in bands of 8 token tiles, whose
// operands the XCD's L2 then holds.
__device__ __forceinline__ void tile_of(const LinearArgs& a, int BT, int BN, int64_t& t0, int& n0)
{
    const int nwg = a.tiles_t * a.tiles_n, b = blockIdx.x;
    const int q = nwg >> 3, r = nwg & 7, x = b & 7;
    const int id = x * q + (x < r ? x : r) + (b >> 3);
    const int per = 8 * a.tiles_n, band = id / per, in = id - band * per;
    const int left = a.tiles_t - band * 8, high = left < 8 ? left : 8;
    t0 = (int64_t)(band * 8 + in % high) * BT;
    n0 = in / high * BN;
}

template <int BT, int BN, int WT, int WN, int KB, int ST, bool EMBED, bool UNAL>
__global__ __launch_bounds__(WT* WN * 64) void tile_kernel(LinearArgs a)
{
    typedef Tile<BT, BN, WT, WN, KB, ST, EMBED, UNAL> C;
    __shared__ __align__(1024) uint8_t ring[ST * C::kStage];
    __shared__ __align__(16) float ws[BN], bs[BN];
    __shared__ double red[EMBED && WN > 1 ? 2 * WN * BT : 1];

    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int wt = wave / WN, wn = wave % WN;

    int64_t t0;
    int n0;
    tile_of(a, BT, BN, t0, n0);
    const int rows_t = (int)(a.T - t0 < BT ? a.T - t0 : BT);
    const int rows_n = a.N - n0 < BN ? a.N - n0 : BN;
    const int8_t* A = a.A + t0 * a.K;
    const int8_t* W = a.W + (int64_t)n0 * a.K;
    for (int i = threadIdx.x; i < BN; i += C::kThreads) {
        ws[i] = i < rows_n ? a.w_scale[n0 + i] : 0.0f;
        bs[i] = a.bias && i < rows_n ? a.bias[n0 + i] : 0.0f;
    }

    i32x16 acc[C::NT][C::TT];
#pragma unroll
    for (int i = 0; i < C::NT; ++i)
#pragma unroll
        for (int j = 0; j < C::TT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    const int a_row = wt * C::TT * 32, w_row = BT + wn * C::NT * 32;

    // The wave's loads: load j covers kRows rows, one chunk per lane. Rows past
    // the end of an operand repeat its last row; what they give is not stored.
    uint32_t voff[C::kPerWave];
    auto row_of = [&](int j) { return (wave * C::kPerWave + j) * C::kRows; };
#pragma unroll
    for (int j = 0; j < C::kPerWave; ++j) {
        const int base = row_of(j), r = base + lane / C::kCpr;
        const bool isA = base < BT;
        const int local = isA ? r : channel_of(r - BT), last = (isA ? rows_t : rows_n) - 1;
        voff[j] = (uint32_t)(local < last ? local : last) * (uint32_t)a.K +
                  (uint32_t)place<KB>(r, lane % C::kCpr) * 16;
    }

    const int nk = UNAL ? 0 : a.K / KB;  // stages filled by direct-to-LDS loads
    if constexpr (!UNAL) {
        const uint32_t ring0 = lds_addr(ring);
        // The order of k does not matter to whole numbers. Rows a multiple of 4 KB
        // apart meet the same few memory channels at one k, so workgroups that read
        // their hidden states from memory start at different ones (100,000 x 4096 to
        // 128 channels 102 us, 121 without).
        const int first = EMBED && (a.K & 4095) == 0 ? (int)(blockIdx.x % (unsigned)nk) : 0;
        auto issue = [&](int i) {
            const int ki = first + i < nk ? first + i : first + i - nk;
            const int8_t* pa = A + (int64_t)ki * KB;
            const int8_t* pw = W + (int64_t)ki * KB;
            const uint32_t at = ring0 + (uint32_t)(i % ST) * C::kStage;
            constexpr int kGroup = C::kPerWave % 4 == 0 && C::kLoads % C::kWaves == 0 && BT % (4 * C::kRows) == 0 ? 4 : 1;
#pragma unroll
            for (int j = 0; j < C::kPerWave; j += kGroup) {
                const int base = row_of(j);
                const uint32_t to = (uint32_t)uniform((int)(at + base * KB));
                if constexpr (kGroup == 4) {
                    if (EMBED && base < BT) dma_lds16_x4<true>(uniform_ptr(pa), &voff[j], to);
                    else dma_lds16_x4<false>(uniform_ptr(base < BT ? pa : pw), &voff[j], to);
                    continue;
                }
                // embeddings: the hidden states pass once, W is read by every workgroup
                if (EMBED && base < BT) dma_lds16_nt(uniform_ptr(pa), voff[j], to);
                else if (C::kLoads % C::kWaves == 0 || base < BT + BN)
                    dma_lds16(uniform_ptr(base < BT ? pa : pw), voff[j], to);
            }
        };
#pragma unroll
        for (int s = 0; s < ST - 1; ++s)
            if (s < nk) issue(s);
        for (int i = 0; i < nk; ++i) {
            // stage i has landed: at most the loads of the ST - 2 later stages are out
            if (ST > 2 && i + ST - 2 < nk) wait_vmcnt<(ST - 2) * C::kPerWave>();
            else wait_vmcnt<0>();
            block_barrier();  // all waves' loads of stage i landed; stage i - 1 is read
            if (i + ST - 1 < nk) issue(i + ST - 1);
            multiply<C, KB>(ring + (i % ST) * C::kStage, w_row, a_row, acc);
        }
    }
    // The rest of k (all of it when rows are not 16-byte aligned) goes through
    // registers, which fill up with zeros past the end of a row. The loads of one
    // stage fly while the stage before it is multiplied.
    constexpr int kChunks = ((BT + BN) * C::kCpr + C::kThreads - 1) / C::kThreads;
    const int8_t* src[kChunks];
    int chunk[kChunks], to[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int c = j * C::kThreads + threadIdx.x, r = c / C::kCpr;
        const bool isA = r < BT;
        const int local = isA ? r : channel_of(r - BT), last = (isA ? rows_t : rows_n) - 1;
        src[j] = (isA ? A : W) + (int64_t)(local < last ? local : last) * a.K;
        chunk[j] = c % C::kCpr * 16;
        to[j] = r < BT + BN ? r * KB + place<KB>(r, c % C::kCpr) * 16 : -1;
    }
    i32x4 part[kChunks];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
            if (to[j] >= 0) part[j] = load16<UNAL>(src[j], k0 + chunk[j], a.K);
    };
    if (nk * KB < a.K) fetch(nk * KB);
    for (int k0 = nk * KB, i = nk; k0 < a.K; k0 += KB, ++i) {
        if (i == nk) __syncthreads();  // the last readers of the direct stages are done
        uint8_t* buf = ring + (i & 1) * C::kStage;
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
            if (to[j] >= 0) *(i32x4*)(buf + to[j]) = part[j];
        if (k0 + KB < a.K) fetch(k0 + KB);
        block_barrier();  // stage i is written; stage i - 1, the other buffer, is read
        multiply<C, KB>(buf, w_row, a_row, acc);
    }
    __syncthreads();  // ws and bs are written

    const int half = lane >> 5;
    if constexpr (EMBED) {
        int64_t t[C::TT];
        int slot[C::TT];
        float as[C::TT];
        bool live[C::TT];
#pragma unroll
        for (int j = 0; j < C::TT; ++j) {
            slot[j] = a_row + j * 32 + (lane & 31);
            t[j] = t0 + slot[j];
            live[j] = t[j] < a.T && (!a.mask || a.mask[t[j]]);
            as[j] = live[j] ? a.a_scale[t[j]] : 0.0f;
        }
        embed_rows<C::TT, C::NT, 16, 32, WN>(
            a, [&](auto j, auto b, auto i) { return acc[b][j][(int)i]; },
            [&](int b) { return (wn * C::NT + b) * 32 + half * 16; }, ws, bs, t, as, live, slot, wn, red, BT);
    } else {
        store_tile<C::NT, C::TT>(a, acc, ws, bs, t0, n0, a_row, wn, wave, ring);
    }
}

// ---------------------------------------------------------------------------
// Many tokens through a narrow projection
// ---------------------------------------------------------------------------

// For embeddings of up to NWV x 32 channels of K <= KS x 32 (a multiple of 128)
// the weights fit in registers: each of NWV waves keeps its 32 channels for the
// whole run, and the hidden states stream through an LDS ring of ST stages, 32
// whole rows each, one contiguous piece of memory. Nothing but the states is
// read again and again, each byte once.
template <int KS, int NWV, int ST, bool CODES>
__global__ __launch_bounds__(NWV * 64, 2) void stream_kernel(LinearArgs a)
{
    constexpr int kScales = KS * 1024, kMask = kScales + 256, kStage = kMask + 256;
    constexpr int PW = (KS + NWV - 1) / NWV;  // wave-wide loads of rows per wave and stage
    constexpr int kLoads = PW + 2;            // and the tokens' scales and mask
    __shared__ __align__(1024) uint8_t ring[ST * kStage];
    __shared__ __align__(16) float ws[NWV * 32], bs[NWV * 32];
    __shared__ double red[2 * 2 * NWV * 32];
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id(), l = lane & 31, half = lane >> 5;
    const int K = a.K;

    for (int i = threadIdx.x; i < NWV * 32; i += NWV * 64) {
        ws[i] = i < a.N ? a.w_scale[i] : 0.0f;
        bs[i] = a.bias && i < a.N ? a.bias[i] : 0.0f;
    }
    i32x4 w[KS];
    {
        const int n = wave * 32 + channel_of(l);
        const int8_t* row = a.W + (int64_t)(n < a.N ? n : 0) * K;
#pragma unroll
        for (int s = 0; s < KS; ++s) w[s] = load16<false>(row, n < a.N ? s * 32 + half * 16 : K, K);
    }

    // 16-byte chunk c of row r lies at chunk c ^ f(r) of its row, so that 16
    // lanes that read one chunk of consecutive rows meet no bank twice: rows are
    // a multiple of 256 bytes apart, or an odd multiple of 128
    const bool even = (K & 255) == 0;
    auto f = [&](int r) { return even ? r & 15 : (r >> 1) & 7; };
    const int cpr = K / 16, loads = K / 32;
    auto load_of = [&](int j) { return wave * PW + j < loads ? wave * PW + j : loads - 1; };  // a spare load
    uint32_t voff[PW];                                                                        // repeats the last
#pragma unroll
    for (int j = 0; j < PW; ++j) {
        const int p = load_of(j) * 64 + lane, r = p / cpr;
        voff[j] = (uint32_t)(r * K + ((p % cpr) ^ f(r)) * 16);
    }
    const uint32_t ring0 = lds_addr(ring);
    const int count = (a.tiles_t - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;  // tiles of this workgroup
    auto issue = [&](int i) {
        const int64_t t0 = ((int64_t)blockIdx.x + (int64_t)i * gridDim.x) * 32;
        const int last = (int)(a.T - t0 < 32 ? a.T - t0 : 32) - 1;
        const uint32_t to = ring0 + (uint32_t)(i % ST) * kStage;
        const void* src = uniform_ptr(a.A + t0 * K);
#pragma unroll
        for (int j = 0; j < PW; ++j) {
            uint32_t v = voff[j];
            if (last < 31) {  // rows past the end repeat the last one
                const int r = (load_of(j) * 64 + lane) / cpr;
                v -= (uint32_t)((r > last ? r - last : 0) * K);
            }
            dma_lds16_nt(src, v, (uint32_t)uniform((int)(to + load_of(j) * 1024)));
        }
        // every wave brings the 32 scales and mask bytes, so that all count alike
        dma_lds4(uniform_ptr(a.a_scale + t0), (uint32_t)(lane < last ? lane : last) * 4,
                 (uint32_t)uniform((int)(to + kScales)));
        // the aligned words that hold the tile's mask bytes, and only those
        const uintptr_t m = a.mask ? (uintptr_t)(a.mask + t0) : (uintptr_t)(a.a_scale + t0);
        const int words = ((int)(m & 3) + last + 4) >> 2;
        dma_lds4(uniform_ptr((const void*)(m & ~(uintptr_t)3)), (uint32_t)(lane < words ? lane : words - 1) * 4,
                 (uint32_t)uniform((int)(to + kMask)));
    };
    const int mask_at = a.mask ? (int)((uintptr_t)a.mask & 3) : 0;  // tiles start at multiples of 32
    int off[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) off[j] = l * K + ((2 * j + half) ^ f(l)) * 16;

#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
        if (s < count) issue(s);
    // One barrier per tile: it hands over the tile that landed and, with it, the
    // statistics of the tile before, which is normalised and written beside the
    // next one's MFMAs.
    Rows<CODES, 1, 1, 16, 32, NWV> rows{};
    int64_t t[1] = {a.T};  // no tile before the first
    float as[1];
    bool live[1] = {false};
    const int slot[1] = {l};
    i32x16 acc;
    auto sum = [&](auto, auto, auto r) { return acc[(int)r]; };
    auto chan = [&](int) { return wave * 32 + half * 16; };
    auto finish = [&](int i) {
        rows.second(a, sum, chan, ws, bs, t, as, live, red + (i & 1) * (2 * NWV * 32), 32, slot, wave);
    };
    for (int i = 0; i < count; ++i) {
        if (i + ST - 2 < count) wait_vmcnt<(ST - 2) * kLoads>();
        else wait_vmcnt<0>();
        block_barrier();  // all waves' loads of stage i landed; stage i - 1 is read
        const uint8_t* st = ring + (i % ST) * kStage;
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = 0;
        // where K < KS * 32, the last fragments of w are zeros and the bytes they
        // meet are those of other rows
#pragma unroll
        for (int s = 0; s < KS; ++s)
            acc = mfma32<kI8>(w[s], *(const i32x4*)(st + off[s & 7] + (s >> 3) * 256), acc);
        // the next loads follow the MFMAs (73 us for the 360,000 x 768 states, 81
        // with the loads in front of them)
        if (i + ST - 1 < count) issue(i + ST - 1);
        finish(i + 1);
        t[0] = ((int64_t)blockIdx.x + (int64_t)i * gridDim.x) * 32 + l;
        live[0] = t[0] < a.T && (!a.mask || st[kMask + mask_at + l]);
        as[0] = live[0] ? *(const float*)(st + kScales + l * 4) : 0.0f;
        rows.first(sum, chan, ws, bs, as, live);
        rows.put(red + (i & 1) * (2 * NWV * 32), 32, slot, wave);
    }
    block_barrier();
    finish(count - 1);
}

// ---------------------------------------------------------------------------
// A few tokens
// ---------------------------------------------------------------------------

// What few_kernel makes of its sums: products, whole normalised rows, or normalised
// rows whose channels are spread over workgroups (see embed_split).
enum Few : int { kProduct, kWhole, kStats, kFinish };

// TT tiles of 16 tokens x (NW * NPW) tiles of 16 channels per workgroup; NW
// waves side by side over the channels, KW waves over k.
template <int TT, int NPW, int NW, int KW, int MODE, bool UNAL>
__global__ __launch_bounds__(NW* KW * 64) void few_kernel(LinearArgs a)
{
    constexpr bool EMBED = MODE == kWhole, SPLIT = MODE == kStats || MODE == kFinish;
    static_assert(!SPLIT || (NPW == 1 && NW == 1), "one tile of channels");
    constexpr int BN = NW * NPW * 16;
    __shared__ __align__(16) float ws[BN], bs[BN];
    __shared__ __align__(16) i32x4 sums[KW > 1 ? (KW - 1) * NW * NPW * TT * 64 : 1];
    __shared__ double red[EMBED && NW > 1 ? 2 * NW * TT * 16 : 1];
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int kw = wave / NW, nw = wave % NW;
    const int n0 = EMBED ? 0 : (int)blockIdx.x * BN;
    const int64_t t0 = (int64_t)(EMBED ? blockIdx.x : blockIdx.y) * (TT * 16);
    const int row = lane & 15, quarter = lane >> 4;

    for (int i = threadIdx.x; i < BN; i += NW * KW * 64) {
        ws[i] = n0 + i < a.N ? a.w_scale[n0 + i] : 0.0f;
        bs[i] = a.bias && n0 + i < a.N ? a.bias[n0 + i] : 0.0f;
    }
    const int8_t* wp[NPW];
    const int8_t* ap[TT];
#pragma unroll
    for (int p = 0; p < NPW; ++p) {
        const int n = n0 + (nw * NPW + p) * 16 + row;
        wp[p] = a.W + (int64_t)(n < a.N ? n : a.N - 1) * a.K;
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = t0 + j * 16 + row;
        ap[j] = a.A + (t < a.T ? t : a.T - 1) * a.K;
    }
    float as[TT];  // loaded beside the first rows
    bool live[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = t0 + j * 16 + row;
        const bool in = t < a.T && kw == 0;
        as[j] = in ? a.a_scale[t] : 0.0f;
        live[j] = in && (MODE == kProduct || !a.mask || a.mask[t]);
    }
    i32x4 acc[NPW][TT];
#pragma unroll
    for (int p = 0; p < NPW; ++p)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[p][j] = i32x4{};

    const int steps = (a.K + 63) / 64, per = (steps + KW - 1) / KW;
    const int s1 = (kw + 1) * per < steps ? (kw + 1) * per : steps;
    constexpr int U = TT + NPW <= 2 ? 8 : TT + NPW <= 4 ? 4 : 2;  // steps whose loads fly together
    for (int s = kw * per; s < s1; s += U) {
        i32x4 w[U][NPW], x[U][TT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = s + u < s1 ? (s + u) * 64 + quarter * 16 : a.K;  // k >= K gives zeros
#pragma unroll
            for (int p = 0; p < NPW; ++p) w[u][p] = load16<UNAL>(wp[p], k, a.K);
#pragma unroll
            for (int j = 0; j < TT; ++j) x[u][j] = load16<UNAL>(ap[j], k, a.K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int p = 0; p < NPW; ++p)
#pragma unroll
                for (int j = 0; j < TT; ++j)
                    acc[p][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][p], x[u][j], acc[p][j], 0, 0, 0);
    }
    if constexpr (KW > 1) {
        if (kw > 0) {
#pragma unroll
            for (int p = 0; p < NPW; ++p)
#pragma unroll
                for (int j = 0; j < TT; ++j) sums[((((kw - 1) * NW + nw) * NPW + p) * TT + j) * 64 + lane] = acc[p][j];
        }
    }
    __syncthreads();
    if constexpr (KW > 1) {
        if (kw == 0) {
            for (int o = 0; o < KW - 1; ++o) {
#pragma unroll
                for (int p = 0; p < NPW; ++p)
#pragma unroll
                    for (int j = 0; j < TT; ++j) acc[p][j] += sums[(((o * NW + nw) * NPW + p) * TT + j) * 64 + lane];
            }
        }
    }
    if constexpr (EMBED) {
        // the waves of other k parts only keep the barriers: they hold no rows
        int64_t t[TT];
        int slot[TT];
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            slot[j] = j * 16 + row;
            t[j] = kw == 0 ? t0 + slot[j] : a.T;
            if (!live[j]) as[j] = 0.0f;
        }
        embed_rows<TT, NPW, 4, 16, NW>(
            a, [&](auto j, auto b, auto i) { return acc[b][j][(int)i]; },
            [&](int b) { return (nw * NPW + b) * 16 + quarter * 4; }, ws, bs, t, as, live, slot, kw == 0 ? nw : -1, red,
            TT * 16);
    } else if constexpr (SPLIT) {
        if (kw > 0) return;
        int64_t t[TT];
        int slot[TT] = {};
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            t[j] = t0 + j * 16 + row;
            if (!live[j]) as[j] = 0.0f;
        }
        auto sum = [&](auto j, auto, auto i) { return acc[0][j][(int)i]; };
        auto local = [&](int) { return quarter * 4; };
        const int64_t es = a.out == kI8 ? 1 : a.out == kF32 ? 4 : 2;
        auto go = [&](auto& rows) {
            rows.first(sum, local, ws, bs, as, live);
            if constexpr (MODE == kStats) rows.put(nullptr, 0, slot, 0);
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                if (t[j] >= a.T) continue;
                double* stat = (double*)((char*)a.Y + (t[j] * a.N + n0) * es);
                if constexpr (MODE == kStats) {
                    if (quarter == 0) {
                        stat[0] = rows.top[j];
                        stat[1] = rows.ss[j];
                    }
                } else {
                    rows.top[j] = stat[0];
                    rows.ss[j] = stat[1];
                }
            }
            if constexpr (MODE == kFinish) {
                // the whole wave has its statistics before any lane overwrites them
                __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
                lds_fence();
                LinearArgs at = a;  // channels are counted from n0 in ws and bs
                at.Y = (char*)a.Y + n0 * es;
                rows.second(at, sum, local, ws, bs, t, as, live, nullptr, 0, slot, n0 == 0 ? 0 : -1);
            }
        };
        if (a.out == kI8) {
            Rows<true, TT, 1, 4, 16, 1> rows;
            go(rows);
        } else {
            Rows<false, TT, 1, 4, 16, 1> rows;
            go(rows);
        }
    } else {
        if (kw > 0) return;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int64_t t = t0 + j * 16 + row;
            if (t >= a.T) continue;
#pragma unroll
            for (int p = 0; p < NPW; ++p) {
                const int n = (nw * NPW + p) * 16 + quarter * 4;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = scaled(acc[p][j][e], as[j], ws[n + e], bs[n + e]);
                store_run<4>(a.Y, a.out, t, n0 + n, a.N, y);
            }
        }
    }
}

// Joins the statistics that N / 16 workgroups left in each row (lane r those of
// channels 16 r ..) and leaves the row's in every one of their places. A wave
// takes a row.
__global__ __launch_bounds__(256) void join_kernel(LinearArgs a)
{
    const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    const int r = threadIdx.x & 63;
    if (t >= a.T) return;
    const int64_t es = a.out == kI8 ? 1 : a.out == kF32 ? 4 : 2;
    double* stat = (double*)((char*)a.Y + (t * a.N + r * 16) * es);
    const bool has = r * 16 < a.N;
    double top = has ? stat[0] : 0.0, ss = has ? stat[1] : 0.0;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        top = __builtin_fmax(top, xor_lane(top, m));
        ss += xor_lane(ss, m);
    }
    if (has) {
        stat[0] = top;
        stat[1] = ss;
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

int64_t tiles(int64_t n, int b) { return (n + b - 1) / b; }

template <int BT, int BN, int WT, int WN, int KB, int ST, bool EMBED, bool UNAL>
void run_tiles(LinearArgs a, hipStream_t stream)
{
    a.tiles_t = (int32_t)tiles(a.T, BT);
    a.tiles_n = (int32_t)tiles(a.N, BN);
    hipLaunchKernelGGL((tile_kernel<BT, BN, WT, WN, KB, ST, EMBED, UNAL>), dim3((unsigned)(a.tiles_t * a.tiles_n)),
                       dim3(WT * WN * 64), 0, stream, a);
}

template <int TT, int NPW, int NW, int KW, int MODE>
void run_few(const LinearArgs& a, hipStream_t stream)
{
    const unsigned over_t = (unsigned)tiles(a.T, TT * 16);
    const dim3 grid = MODE == kWhole ? dim3(over_t) : dim3((unsigned)tiles(a.N, NW * NPW * 16), over_t);
    const dim3 block(NW * KW * 64);
    if (a.K % 16 == 0) hipLaunchKernelGGL((few_kernel<TT, NPW, NW, KW, MODE, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((few_kernel<TT, NPW, NW, KW, MODE, true>), grid, block, 0, stream, a);
}

// Tiles by how many the launch has (median us of N = K = 4096 bf16 outputs with
// 256 x 256 / 128 x 128 / 64 x 128 / 64 x 64 tiles):
//   T = 8192  117 / 132 / 168 / 208     2048   48 /  36 /  44 /  52
//   T = 4096   61 /  68 /  84 / 101     1024   48 /  25 /  23 /  28
//   T =  512   46 /  23 /  17 /  16       96   43 /  23 /  16 /  12
// One 256 x 256 tile fills a CU, two or more of the smaller ones share it. Up to
// 32 tokens the direct form is ahead (32 tokens 8.8 against 11.1 us, 16 6.6
// against 11.1; 64 tokens 14.2 against 11.2).
template <bool UNAL>
void linear_tiles(const LinearArgs& a, hipStream_t stream)
{
    const int64_t cus = device_cu_count();
    if (tiles(a.T, 256) * tiles(a.N, 256) >= cus) run_tiles<256, 256, 2, 4, 128, 2, false, UNAL>(a, stream);
    else if (tiles(a.T, 128) * tiles(a.N, 128) >= 2 * cus) run_tiles<128, 128, 2, 2, 128, 2, false, UNAL>(a, stream);
    else if (!UNAL && tiles(a.T, 64) * tiles(a.N, 128) >= 2 * cus)
        run_tiles<64, 128, 2, 2, 128, 3, false, false>(a, stream);
    else run_tiles<64, 64, 2, 2, 128, UNAL ? 2 : 4, false, UNAL>(a, stream);
}

void linear_once(const LinearArgs& a, hipStream_t stream)
{
    if (a.T <= 16) run_few<1, 1, 1, 8, kProduct>(a, stream);
    else if (a.T <= 32) run_few<2, 1, 1, 8, kProduct>(a, stream);
    else if (a.K % 16 == 0) linear_tiles<false>(a, stream);
    else linear_tiles<true>(a, stream);
}

// Every workgroup holds whole rows, so the tile's tokens shrink as the channels
// grow. Up to 128 channels two workgroups of 128 tokens share a CU: 200,000 tokens
// of 2048 to 128 channels take 111 us, 129 with one of 256 tokens, 145 with
// 64-byte steps of k; to 256 channels 156 us with 256 tokens, 193 with 128.
template <bool UNAL>
void embed_tiles(const LinearArgs& a, hipStream_t stream)
{
    if (a.N <= 128) run_tiles<128, 128, 4, 1, 128, 2, true, UNAL>(a, stream);
    else if (a.N <= 256) run_tiles<256, 256, 4, 2, 128, 2, true, UNAL>(a, stream);
    else if (a.N <= 512) run_tiles<64, 512, 2, 4, 128, 2, true, UNAL>(a, stream);
    else if (a.N <= 768) run_tiles<64, 768, 1, 8, 64, 2, true, UNAL>(a, stream);
    else run_tiles<64, 1024, 1, 8, 64, 2, true, UNAL>(a, stream);
}

template <int KS, int NWV, int ST>
void run_stream(LinearArgs a, hipStream_t stream)
{
    a.tiles_t = (int32_t)tiles(a.T, 32);
    const int64_t most = (int64_t)device_cu_count() * (8 / NWV);  // 8 waves on each CU
    const dim3 grid((unsigned)(a.tiles_t < most ? a.tiles_t : most)), block(NWV * 64);
    if (a.out == kI8) hipLaunchKernelGGL((stream_kernel<KS, NWV, ST, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((stream_kernel<KS, NWV, ST, false>), grid, block, 0, stream, a);
}

// The ring's stages: 72 KB a workgroup where two share a CU's LDS, 150 KB for one.
bool stream_ok(const LinearArgs& a) { return a.N <= 256 && a.K <= 1024 && a.K % 128 == 0; }
void embed_stream(const LinearArgs& a, hipStream_t stream)
{
    if (a.N <= 128) {
        if (a.K <= 256) run_stream<8, 4, 6>(a, stream);
        else if (a.K <= 512) run_stream<16, 4, 4>(a, stream);
        else if (a.K <= 768) run_stream<24, 4, 3>(a, stream);
        else run_stream<32, 4, 2>(a, stream);
    } else {
        if (a.K <= 256) run_stream<8, 8, 6>(a, stream);
        else if (a.K <= 512) run_stream<16, 8, 6>(a, stream);
        else if (a.K <= 768) run_stream<24, 8, 5>(a, stream);
        else run_stream<32, 8, 4>(a, stream);
    }
}

// Few tokens, many weights: one CU fills at about 70 B/ns, so one workgroup per
// block of rows would take W's bytes at that rate. Here every tile of 16 channels
// has a workgroup: the first launch leaves the tile's statistics of each row in the
// 16 bytes or more of E that the tile will fill, the second joins a row's, the
// third forms the sums again (W comes from the caches then) and overwrites its own
// place. 32 tokens of 1024 to 1024 channels take 10.5 us, 27.5 in tiles of whole
// rows; of 4096 to 128 17.6 us, 30.9 in the direct form. Three launches cost about
// 5 us more than one, so it takes over 160,000 weights to pay (1000 to 128 channels
// 10.7 against 7.2 us, 1536 to 128 11.2 against 13.6), beyond 256 channels, where
// the other choice is tiles, any number (64 to 512 channels 8.5 against 8.6 us, to
// 1024 8.6 against 13.7). From 1024 tokens on the tiles are ahead (768 to 768
// channels 20.0 against 22.4 us; 512 tokens 19.5 against 14.8).
constexpr int64_t kSplitTokens = 512, kSplitWeights = 160000;
bool split_ok(const LinearArgs& a)
{
    return a.T <= kSplitTokens && a.N % 16 == 0 && (a.N > 256 || (int64_t)a.N * a.K > kSplitWeights);
}
void embed_split(const LinearArgs& a, hipStream_t stream)
{
    if (a.T <= 16) run_few<1, 1, 1, 8, kStats>(a, stream);
    else run_few<2, 1, 1, 8, kStats>(a, stream);
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)tiles(a.T, 4)), dim3(256), 0, stream, a);
    if (a.T <= 16) run_few<1, 1, 1, 8, kFinish>(a, stream);
    else run_few<2, 1, 1, 8, kFinish>(a, stream);
}

// The streamed form where it fits, at any number of tokens (32 to 4096 tokens of
// 768 to 128 channels 6.4 to 7.1 us, direct form 8.5 to 9.1, tiles 8.9 to 11.8; a
// single token 6.4 in both the first). Elsewhere few tokens spread their channels
// over workgroups if the weights are many, or take the direct form up to 256
// channels (4096 tokens of 2048 to 128 channels 18.0 us, tiles 20.5; 1024 tokens
// 17.4, tiles 15.2), and tiles beyond.
void embed_once(const LinearArgs& a, hipStream_t stream)
{
    if (stream_ok(a)) return embed_stream(a, stream);
    if (split_ok(a)) return embed_split(a, stream);
    if (a.T <= 4096 && a.N <= 128) return run_few<1, 1, 8, 2, kWhole>(a, stream);
    if (a.T <= 4096 && a.N <= 256) return run_few<1, 1, 16, 1, kWhole>(a, stream);
    if (a.K % 16 == 0) embed_tiles<false>(a, stream);
    else embed_tiles<true>(a, stream);
}

// One launch covers at most `step` rows, so that a grid's threads stay below
// 2^32; the rows are independent.
template <typename F>
hipError_t by_rows(LinearArgs a, int64_t step, F once)
{
    const int64_t es = a.out == kF32 ? 4 : a.out == kI8 ? 1 : 2;
    for (int64_t left = a.T; left > 0; left -= step) {
        a.T = left < step ? left : step;
        once(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.A += step * a.K;
        a.a_scale += step;
        if (a.mask) a.mask += step;
        a.Y = (char*)a.Y + step * a.N * es;
        if (a.y_scale) a.y_scale += step;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_linear_i8(LinearArgs a, hipStream_t stream)
{
    // N is at most 2^26, so 256 rows make at most 2^22 tiles of 64 x 64
    int64_t step = (int64_t)1 << 24;
    while (step > 256 && tiles(step, 64) * tiles(a.N, 64) > (1 << 22)) step /= 2;
    return by_rows(a, step, [&](const LinearArgs& x) { linear_once(x, stream); });
}

hipError_t launch_embed_i8(LinearArgs a, hipStream_t stream)
{
    return by_rows(a, (int64_t)1 << 26, [&](const LinearArgs& x) { embed_once(x, stream); });
}

}  // namespace maxsim
