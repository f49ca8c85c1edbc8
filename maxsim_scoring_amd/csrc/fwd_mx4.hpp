#pragma once

// Cross-product MaxSim of microscaled 4-bit queries and documents for gfx950,
// with masks, optional argmax and queries of any length.
//
//   score[i,j] = sum_s max_t sum_b 2^(eq[s,b] + ed[t,b]) <Q[s,b], D[t,b]>
//
// The tile is transposed as in the other forwards, S^T = D . Q^T: MFMA rows are
// document tokens, columns query tokens, so the max over tokens stays inside a
// lane until the document ends. The block-scaled MFMA takes codes and exponents as
// they are stored; a token of 128 channels is 64 bytes of codes and one word of
// exponents, of which lane half h takes blocks 2 h and 2 h + 1 of every four.
//
// A unit of work is one wave: up to NTW tiles of 32 query tokens, held in
// registers, against a range of documents, whose tokens go straight from memory
// to registers, P tiles of 32 ahead and across the ends of documents. The tokens of a
// unit stay in the caches for the other units of its range, which follow it on the
// same XCD. Queries of more than NTW tiles are split over the four waves of a
// workgroup, which leave their sums in LDS to be added in order; otherwise waves share
// nothing. Queries of up to 16 tokens share a tile, in slots of a power of two columns.
//
// Masked tokens cost nothing per query tile: the accumulator starts at -inf in
// their rows, and their exponents become 0, which is 2^-127. So a NaN among them is
// not seen (codes are finite whatever they are), and their products stay finite
// beside any query block that is not NaN: an exponent of 2^0 would let the largest
// ones overflow to +inf, and their sum with -inf is NaN. A range's mask becomes bits
// in LDS first, so that the masked tail of a padded document is not read at all.
//
// One query of 32 tokens over 50,000 documents of 180, a quarter masked, 128 channels:
// 94 us, 468 MB at 5.0 TB/s (without a mask 612 MB at 5.45, the rate of a copy). 32
// queries over 1000 pages of 1024 tokens: 66 us, 4.1 PFLOP/s of the 4.6 to 5.1 that a
// loop of these MFMAs alone reaches; 7.5 us for 5 queries over 333 short documents, a
// launch and a few chains of loads. Loads that bypass the caches were slower (98 us
// against 94, 256 channels 117 against 71): later chunks of a line come from L1.
#include "mx4_common.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

constexpr int kWaves = 4;
constexpr int kMaskWords = 512;  // of a wave: the bits of 16,384 tokens
constexpr int kSplitDocs = 256;  // documents whose sums the waves of a split query leave in LDS

typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

// One bit for each of the 4 bytes of x that is not 0.
__device__ __forceinline__ uint32_t byte_bits(uint32_t x)
{
    x |= x >> 4;
    x |= x >> 2;
    x |= x >> 1;
    return (((x & 0x01010101u) * 0x01020408u) >> 24) & 0xfu;
}

// Bits of mask bytes p[0 .. n - 1], n <= 32.
__device__ __forceinline__ uint32_t mask_word(const uint8_t* p, int n)
{
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (4 * k + 4 <= n) bits |= byte_bits(*(const u32_any*)(p + 4 * k)) << (4 * k);
    for (int i = n & ~3; i < n; ++i) bits |= (uint32_t)(p[i] != 0) << i;
    return bits;
}

__device__ __forceinline__ float vmax(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, row16_sum(v));
    return (as_float(__builtin_amdgcn_readlane(b, 0)) + as_float(__builtin_amdgcn_readlane(b, 16))) +
           (as_float(__builtin_amdgcn_readlane(b, 32)) + as_float(__builtin_amdgcn_readlane(b, 48)));
}

// The largest of 16 values and m, NaN where one is.
__device__ __forceinline__ float max16(const f32x16& v, float m)
{
#pragma unroll
    for (int q = 0; q < 16; q += 2) m = vmax(vmax(m, v[q]), v[q + 1]);
    return m;
}

// 4 G blocks of one token of this lane's half: blocks 4 g + 2 h + k in code[2 g + k],
// exponents in bytes 0 and 1 of scale[g].
template <int G>
struct Token {
    i32x4 code[2 * G];
    int scale[G];
};

// FAST: nb is 4 G and the exponents of a token are aligned words.
// base, sbase: the first token of the tile (uniform); row: this lane's. Blocks behind
// the last one repeat it with exponent 2^0: QUERY makes their codes zeros, so that
// they add nothing, whatever the document's are.
template <int G, bool FAST, bool QUERY>
__device__ __forceinline__ void load_token(Token<G>& t, const uint8_t* base, const uint8_t* sbase, int row, int h, int nb)
{
    const uint32_t at = (uint32_t)(row * nb) * 16, sat = (uint32_t)(row * nb);
    static_for<0, G>([&](auto g) {
        if constexpr (FAST) {
            t.code[2 * g] = *(const i32x4*)(base + (at + (4 * g + 2 * h) * 16));
            t.code[2 * g + 1] = *(const i32x4*)(base + (at + (4 * g + 2 * h + 1) * 16));
            t.scale[g] = *(const int*)(sbase + (sat + 4 * g));
        } else {
            const int b = 4 * g + 2 * h;  // and b + 1
            static_for<0, 2>([&](auto k) {
                const int c = b + k < nb ? b + k : nb - 1;
                t.code[2 * g + k] = *(const i32x4*)(base + (at + c * 16));
                if (QUERY) t.code[2 * g + k] = b + k < nb ? t.code[2 * g + k] : i32x4{};
            });
            // both exponents in one load: that of a last block alone comes with the one before
            uint32_t s;
            if (nb == 1) s = sbase[sat];
            else {
                const int c = b < nb - 2 ? b : nb - 2;
                s = *(const u16_any*)(sbase + (sat + c));
                s >>= b == nb - 1 ? 8 : 0;
            }
            s = b + 1 < nb ? s : b < nb ? (s & 0xffu) | 0x7f00u : 0x7f7fu;
            t.scale[g] = (int)s;
        }
    });
}
// The exponents of this lane's half moved to the low bytes.
template <int G, bool FAST>
__device__ __forceinline__ void place_scales(Token<G>& t, int h)
{
    if constexpr (FAST) {
#pragma unroll
        for (int g = 0; g < G; ++g) t.scale[g] = (int)((uint32_t)t.scale[g] >> (16 * h));
    }
}

// Workgroup b of n runs on XCD b % 8: each XCD takes a run of consecutive units.
__device__ __forceinline__ int xcd_order(int b, int n)
{
    const int full = n >> 3, rem = n & 7, xcd = b & 7;
    return xcd * full + (xcd < rem ? xcd : rem) + (b >> 3);
}

// How a query's tokens lie in the unit's tiles.
enum {
    kWhole,   // whole queries of one or more tiles each
    kSplit,   // one query over the waves of a workgroup
    kPacked,  // queries of up to 16 tokens share tiles, in slots of a power of two
};

template <int G, int NTW, int P, bool ARGMAX, bool FAST, int MODE>
__global__ __launch_bounds__(kWaves * 64) void fwd_mx4_kernel(Mx4FwdArgs a)
{
    constexpr bool SPLIT = MODE == kSplit, PACKED = MODE == kPacked;
    __shared__ uint32_t mask_lds[kWaves][kMaskWords];
    __shared__ float part[SPLIT ? kWaves : 1][SPLIT ? kSplitDocs : 1];

    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id(), col = lane & 31, h = lane >> 5;
    uint32_t* const my_mask = mask_lds[wave];

    const int wg = xcd_order(blockIdx.x, gridDim.x);
    const int64_t unit = SPLIT ? wg : (int64_t)wg * kWaves + wave;
    if (unit >= (int64_t)a.nqb * a.nranges) return;  // (the whole workgroup, if SPLIT)
    const int qb = (int)(unit % a.nqb);
    const int64_t r = unit / a.nqb;
    const int d0 = uniform((int)(r * a.Nd / a.nranges)), d1 = uniform((int)((r + 1) * a.Nd / a.nranges));
    if (d0 >= d1) return;

    const int Lq = (int)a.Lq, Ld = (int)a.Ld, nb = a.nb;
    const int tiles = (Ld + 31) / 32;  // of a document
    const bool in_lds = a.d_mask && tiles <= kMaskWords;
    int batch = in_lds ? kMaskWords / tiles : 0x7fffffff;  // documents whose mask LDS holds
    if (SPLIT) batch = batch < kSplitDocs ? batch : kSplitDocs;
    // queries of this unit; tiles of one
    const int i0 = uniform(qb * a.qpw);
    const int nq = uniform((int)(a.Nq - i0 < a.qpw ? a.Nq - i0 : a.qpw));
    const int ntq = a.ntq;
    const int lq = a.log2_qslot, qpt = 32 >> lq;  // columns of a packed query, queries of a tile

    // a split query takes a pass for each kWaves * NTW of its tiles
    for (int q0 = 0; q0 == 0 || (SPLIT && q0 < ntq); q0 += kWaves * NTW) {
        const int first = SPLIT ? q0 + wave * NTW : 0;  // this wave's first tile of a split query
        // ---- the unit's query tiles --------------------------------------------
        Token<G> q[NTW];
        uint32_t live = 0;  // bit n: this lane's column of tile n exists and counts
        static_for<0, NTW>([&](auto n) {
            if constexpr (PACKED) {
                const int qi = n * qpt + (col >> lq), s = col & ((1 << lq) - 1);
                const int64_t base = (int64_t)i0 * Lq;
                const int row = (qi < nq ? qi : nq - 1) * Lq + (s < Lq ? s : Lq - 1);
                load_token<G, FAST, true>(q[n], a.Q + base * nb * 16, a.q_scale + base * nb, row, h, nb);
                place_scales<G, FAST>(q[n], h);
                live |= (uint32_t)(qi < nq && s < Lq && (!a.q_mask || a.q_mask[base + row])) << n;
            } else {
                // tile n is tile n % ntq of query n / ntq, or tile first + n of the one query
                const int qi = SPLIT ? 0 : n / ntq, qt = SPLIT ? first + n : n % ntq;
                const bool tile_in = qi < nq && qt < ntq;
                const int64_t i = i0 + (tile_in ? qi : 0);
                const int t0 = tile_in ? qt * 32 : 0, s = t0 + col;
                const int row = s < Lq ? col : Lq - 1 - t0;
                const int64_t tok = i * Lq + t0;
                load_token<G, FAST, true>(q[n], a.Q + tok * nb * 16, a.q_scale + tok * nb, row, h, nb);
                place_scales<G, FAST>(q[n], h);
                const bool on = tile_in && s < Lq && (!a.q_mask || a.q_mask[i * Lq + s]);
                live |= (uint32_t)on << n;
            }
        });

        float m[NTW];
        int best[ARGMAX ? NTW : 1];
        auto reset = [&] {
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
                m[n] = -__builtin_inff();
                if (ARGMAX) best[n] = 0;
            }
        };
        reset();
        bool any = false;  // a token of the document counts

        for (int64_t first_doc = d0; first_doc < d1; first_doc += batch) {
            const int b0 = (int)first_doc, b1 = d1 - b0 < batch ? d1 : b0 + batch;
            if (in_lds) {
                const int words = (b1 - b0) * tiles;
                for (int w = lane; w < words; w += 64) {
                    const int64_t doc = b0 + w / tiles;
                    const int t0 = w % tiles * 32;
                    my_mask[w] = mask_word(a.d_mask + doc * Ld + t0, Ld - t0 < 32 ? Ld - t0 : 32);
                }
                lds_fence();
                __builtin_amdgcn_wave_barrier();
            }

            auto first_token = [&](int doc) {  // that counts, 0 if none does
                for (int t0 = 0; t0 < Ld; t0 += 64) {
                    const uint64_t some = __ballot(lane < Ld - t0 && a.d_mask[(int64_t)doc * Ld + t0 + lane]);
                    if (some) return t0 + __builtin_ctzll(some);
                }
                return 0;
            };

            // Sums of a finished document, tiles in order. Both halves of a wave hold the
            // maxima of 32 columns, over different rows: the halves of two tiles are swapped so
            // that one maximum joins both, the first tile's in the low half.
            auto finish = [&](int doc) __attribute__((always_inline)) {
                int i = i0, at = 0;  // the query of tile n, and which of its tiles that is
                float sums = 0.0f;   // of this lane's columns of the query's tiles so far
                auto put = [&](int n, int idx) {
                    if constexpr (PACKED) {
                        const int qi = n * qpt + (col >> lq), s = col & ((1 << lq) - 1);
                        if (qi < nq && s < Lq) a.argmax[((int64_t)(i0 + qi) * a.Nd + doc) * Lq + s] = idx;
                    } else {
                        const int s = (SPLIT ? first + n : at) * 32 + col;
                        if (s < Lq) a.argmax[(i * a.Nd + doc) * Lq + s] = idx;
                    }
                };
                static_for<0, (NTW + 1) / 2>([&](auto pair) {
                    constexpr int n = 2 * pair, n2 = n + 1 < NTW ? n + 1 : n;
                    if (PACKED && n * qpt >= nq) return;
                    if (!SPLIT && !PACKED && i >= i0 + nq) return;
                    if (SPLIT && first + n >= ntq) return;
                    float v;
                    if constexpr (n2 > n) {
                        const auto both = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, m[n]),
                                                                           __builtin_bit_cast(uint32_t, m[n2]), false, false);
                        v = vmax(as_float(both[0]), as_float(both[1]));
                    } else {
                        v = vmax(m[n], shfl_xor_f(m[n], 32));
                    }
                    const bool lost = ARGMAX && v == -__builtin_inff();
                    const bool mine = (live >> (n2 > n && h ? n2 : n)) & 1;
                    v = any && mine && (n2 > n || h == 0) ? v : 0.0f;
                    if constexpr (ARGMAX) {
                        // the lower index of equal maxima
                        static_for<n, n2 + 1>([&](auto k) {
                            const float o = shfl_xor_f(m[k], 32);
                            const int oi = shfl_xor_i(best[k], 32);
                            best[k] = o > m[k] || (o == m[k] && oi < best[k]) ? oi : best[k];
                        });
                        // where all that count are at -inf (products that overflow), the first of them
                        if (__builtin_expect(__any(lost), 0)) {
                            const int first = a.d_mask ? first_token(doc) : 0;
                            static_for<n, n2 + 1>([&](auto k) {
                                best[k] = vmax(shfl_xor_f(m[k], 32), m[k]) == -__builtin_inff() ? first : best[k];
                            });
                        }
                    }
                    if constexpr (MODE != kWhole && ARGMAX) {
                        if (h == 0) put(n, best[n]);
                        if (n2 > n && h == 0) put(n2, best[n2]);
                    }
                    if constexpr (SPLIT) {
                        sums += v;  // (tiles behind the last one have no column that counts)
                    } else if constexpr (PACKED) {
                        if (lq > 0) v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
                        if (lq > 1) v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
                        if (lq > 2) v = dpp_add<0x141>(v);  // row_half_mirror
                        if (lq > 3) v = dpp_add<0x140>(v);  // row_mirror
                        const int qi = (h ? n2 : n) * qpt + (col >> lq);
                        if ((col & ((1 << lq) - 1)) == 0 && qi < nq && (n2 > n || h == 0))
                            a.scores[(int64_t)(i0 + qi) * a.Nd + doc] = v;
                    } else {
                        static_for<n, n2 + 1>([&](auto k) {
                            if (i >= i0 + nq) return;
                            if constexpr (ARGMAX) {
                                if (h == 0) put(k, best[k]);
                            }
                            // the pair's low half is tile n, its high half tile n2
                            sums += (k == n) == (h == 0) ? v : 0.0f;
                            if (++at == ntq) {
                                const float sum = wave_sum(sums);
                                if (lane == 0) a.scores[i * a.Nd + doc] = sum;
                                sums = 0.0f;
                                at = 0;
                                ++i;
                            }
                        });
                    }
                });
                if constexpr (SPLIT) {
                    const float sum = wave_sum(sums);
                    if (lane == 0) part[wave][doc - b0] = sum;
                }
                reset();
                any = false;
            };

            // ---- the stream of tiles ---------------------------------------------
            struct Slot {
                Token<G> t;
                uint32_t bits;      // tokens of the tile that count
                int doc, tile;
                bool last, valid;   // the document's last tile; there is a tile
            } slot[P];
            int doc = b0 - 1, tile = 0, count = 0;  // the tile issued last, tiles of its document
            uint32_t words = 0;  // this lane's of 64 mask words of doc
            const uint8_t* codes = a.D + (int64_t)b0 * Ld * nb * 16;  // of the tile issued last
            const uint8_t* scales = a.d_scale + (int64_t)b0 * Ld * nb;
            auto issue = [&](Slot& s) __attribute__((always_inline)) {
                ++tile;
                codes += 32 * 16 * nb;
                scales += 32 * nb;
                if (tile >= count) {  // the next document with a token
                    for (;;) {
                        if (++doc >= b1) {
                            doc = b1;  // stays behind the end; the tile read is the first one's
                            break;
                        }
                        count = tiles;
                        if (in_lds) {
                            count = 0;
                            for (int w0 = 0; w0 < tiles; w0 += 64) {
                                const uint32_t w = w0 + lane < tiles ? my_mask[(doc - b0) * tiles + w0 + lane] : 0;
                                const uint64_t some = __ballot(w != 0);
                                if (some) count = w0 + 64 - __builtin_clzll(some);
                                if (w0 == 0) words = w;
                            }
                        }
                        if (count > 0) break;
                        // nothing to score
                        if constexpr (SPLIT) {
                            if (lane == 0) part[wave][doc - b0] = 0.0f;
                        }
                        for (int i = i0; i < i0 + nq; ++i) {
                            if (!SPLIT && lane == 0) a.scores[i * a.Nd + doc] = 0.0f;
                            if (ARGMAX)
                                for (int e = lane; e < Lq; e += 64) a.argmax[(i * a.Nd + doc) * Lq + e] = 0;
                        }
                    }
                    tile = 0;
                    if (doc >= b1) count = 0;
                    const int64_t tok = (int64_t)(doc < b1 ? doc : b0) * Ld;
                    codes = a.D + tok * nb * 16;
                    scales = a.d_scale + tok * nb;
                }
                s.valid = doc < b1;
                const int t0 = tile * 32, left = Ld - t0;
                uint32_t bits = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
                if (in_lds && s.valid) {
                    if ((tile & 63) == 0 && tile > 0)
                        words = tile + lane < tiles ? my_mask[(doc - b0) * tiles + tile + lane] : 0;
                    bits = __builtin_amdgcn_readlane(words, tile & 63);
                }
                // rows behind the tile's last token (that counts) repeat it
                const int last = bits ? 31 - __builtin_clz(bits) : 0;
                load_token<G, FAST, false>(s.t, codes, scales, col < last ? col : last, h, nb);
                if (!in_lds && a.d_mask && s.valid)
                    bits = (uint32_t)__ballot(lane < 32 && lane < left && a.d_mask[(int64_t)doc * Ld + t0 + (lane < left ? lane : 0)]);
                s.doc = doc;
                s.tile = tile;
                s.bits = bits;
                s.last = tile + 1 == count;
            };
            auto consume = [&](Slot& s) __attribute__((always_inline)) {
                place_scales<G, FAST>(s.t, h);
                auto fold = [&](auto masked) __attribute__((always_inline)) {
                    f32x16 start;
#pragma unroll
                    for (int e = 0; e < 16; ++e) start[e] = 0.0f;
                    if constexpr (masked) {
                        const bool on = (s.bits >> col) & 1;
                        const uint32_t mine = s.bits >> (4 * h);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            start[e] = (mine >> (8 * (e >> 2) + (e & 3))) & 1 ? 0.0f : -__builtin_inff();
                        // codes are finite whatever they are; an exponent may be NaN
#pragma unroll
                        for (int g = 0; g < G; ++g) s.t.scale[g] = on ? s.t.scale[g] : 0;
                    }
                    static_for<0, NTW>([&](auto n) {
                        f32x16 acc = start;
                        static_for<0, G>([&](auto g) {
                            acc = mfma32_mx4<0, 0>(s.t.code[2 * g], s.t.scale[g], q[n].code[2 * g], q[n].scale[g], acc);
                            acc = mfma32_mx4<1, 1>(s.t.code[2 * g + 1], s.t.scale[g], q[n].code[2 * g + 1], q[n].scale[g], acc);
                        });
                        stay(acc);
                        if constexpr (!ARGMAX) {
                            m[n] = max16(acc, m[n]);
                        } else {
                            const float top = max16(acc, -__builtin_inff());
                            if (top > m[n]) {
                                int row = 0;
#pragma unroll
                                for (int e = 15; e >= 0; --e) row = acc[e] == top ? 8 * (e >> 2) + (e & 3) : row;
                                best[n] = s.tile * 32 + 4 * h + row;
                            }
                            m[n] = vmax(m[n], top);
                        }
                    });
                };
                if (s.bits == 0xffffffffu) fold(std::false_type{});
                else if (s.bits != 0) fold(std::true_type{});
                any |= s.bits != 0;
                if (s.last) finish(s.doc);
            };

            if (SPLIT && first >= ntq) doc = b1;  // no tile of the query is left for this wave
            static_for<0, P>([&](auto p) { issue(slot[p]); });
            while (slot[0].valid) {
                static_for<0, P>([&](auto p) {
                    if (slot[p].valid) {
                        consume(slot[p]);
                        issue(slot[p]);
                    }
                });
            }
            if constexpr (SPLIT) {
                __syncthreads();
                for (int e = threadIdx.x; e < b1 - b0; e += kWaves * 64) {
                    float* out = a.scores + (int64_t)i0 * a.Nd + b0 + e;
                    float sum = part[0][e];
#pragma unroll
                    for (int w = 1; w < kWaves; ++w)
                        if (q0 + w * NTW < ntq) sum += part[w][e];
                    *out = q0 > 0 ? *out + sum : sum;
                }
                __syncthreads();
            }
        }
    }
}

inline int64_t pieces(int64_t n, int b) { return (n + b - 1) / b; }

inline int log2_up(int64_t n)
{
    int l = 0;
    while (((int64_t)1 << l) < n) ++l;
    return l;
}

// The rows that FAST loads take.
template <int G>
bool fast_rows(const Mx4FwdArgs& a)
{
    return a.nb == 4 * G && (((uintptr_t)a.q_scale | (uintptr_t)a.d_scale) & 3) == 0;
}

// WAVES: units that a CU runs at once, 4 for each that a SIMD's registers hold, or
// fewer where more ran slower. ONE: queries of one tile only, where longer ones go to a
// kernel of more tiles.
template <int G, int NTW, int P, int WAVES, bool ONE = false>
void run(Mx4FwdArgs a, hipStream_t stream)
{
    const bool split = !ONE && a.ntq > NTW;
    a.qpw = split ? 1 : NTW / a.ntq;
    a.log2_qslot = 5;
    a.nqb = (int32_t)pieces(a.Nq, a.qpw);
    const int64_t units = (int64_t)device_cu_count() * (split ? WAVES / kWaves : WAVES);
    const int64_t want = units / a.nqb > 0 ? units / a.nqb : 1;
    a.nranges = (int32_t)(want < a.Nd ? want : a.Nd);
    const int64_t total = (int64_t)a.nqb * a.nranges;
    const dim3 grid((unsigned)(split ? total : pieces(total, kWaves))), block(kWaves * 64);
    const bool fast = fast_rows<G>(a);
    // (more query registers beside an argmax's would spill)
#define MAXSIM_MX4_SPLIT(ARGMAX, FAST)                                                                                  \
    do {                                                                                                                \
        if constexpr (!ONE) {                                                                                           \
            if (split) {                                                                                                \
                hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, ARGMAX, FAST, kSplit>), grid, block, 0, stream, a);         \
                break;                                                                                                  \
            }                                                                                                           \
        }                                                                                                               \
        hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, ARGMAX, FAST, kWhole>), grid, block, 0, stream, a);                \
    } while (0)
    if constexpr (NTW < 4 || (NTW == 4 && G < 4)) {
        if (a.argmax && fast) MAXSIM_MX4_SPLIT(true, true);
        else if (a.argmax) MAXSIM_MX4_SPLIT(true, false);
    }
    if (!a.argmax && fast) MAXSIM_MX4_SPLIT(false, true);
    else if (!a.argmax) MAXSIM_MX4_SPLIT(false, false);
#undef MAXSIM_MX4_SPLIT
}

}  // namespace

}  // namespace maxsim
