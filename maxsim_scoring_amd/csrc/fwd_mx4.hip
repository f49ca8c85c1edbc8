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
// to registers, P tiles of 32 ahead and across the ends of documents. Waves share
// nothing, so there is no barrier. The tokens of a unit stay in the caches for the
// other units of its range, which follow it on the same XCD.
//
// Masked tokens cost nothing per query tile: their codes and exponents are
// replaced by zeros and 2^0 (so that a NaN among them is not seen) and the
// accumulator starts at -inf in their rows. A range's mask becomes bits in LDS
// first, so that the masked tail of a padded document is not read at all.
#include "mx4_common.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

constexpr int kWaves = 4;
constexpr int kMaskWords = 512;  // of a wave: the bits of 16,384 tokens

typedef uint32_t u32_any __attribute__((aligned(1)));

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
// base, sbase: the first token of the tile (uniform); row: this lane's.
template <int G, bool FAST>
__device__ __forceinline__ void load_token(Token<G>& t, const uint8_t* base, const uint8_t* sbase, int row, int h, int nb)
{
    const uint32_t at = (uint32_t)(row * nb) * 16, sat = (uint32_t)(row * nb);
    static_for<0, G>([&](auto g) {
        if constexpr (FAST) {
            t.code[2 * g] = *(const i32x4*)(base + (at + (4 * g + 2 * h) * 16));
            t.code[2 * g + 1] = *(const i32x4*)(base + (at + (4 * g + 2 * h + 1) * 16));
            t.scale[g] = *(const int*)(sbase + (sat + 4 * g));
        } else {
            uint32_t s = 0;
            static_for<0, 2>([&](auto k) {
                const int b = 4 * g + 2 * h + k;
                t.code[2 * g + k] = b < nb ? *(const i32x4*)(base + (at + b * 16)) : i32x4{};
                s |= (uint32_t)(b < nb ? sbase[sat + b] : 127) << (8 * k);
            });
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

template <int G, int NTW, int P, bool ARGMAX, bool FAST>
__global__ __launch_bounds__(kWaves * 64) void fwd_mx4_kernel(Mx4FwdArgs a)
{
    __shared__ uint32_t mask_lds[kWaves][kMaskWords];

    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id(), col = lane & 31, h = lane >> 5;
    uint32_t* const my_mask = mask_lds[wave];

    // unit of work: XCD-aware order (workgroup b runs on XCD b % 8)
    const int nblk = gridDim.x, b = blockIdx.x;
    const int full = nblk >> 3, rem = nblk & 7, xcd = b & 7;
    const int64_t unit = (int64_t)(xcd * full + (xcd < rem ? xcd : rem) + (b >> 3)) * kWaves + wave;
    if (unit >= (int64_t)a.nqb * a.nranges) return;
    const int qb = (int)(unit % a.nqb);
    const int64_t r = unit / a.nqb;
    const int64_t d0 = uniform_i64(r * a.Nd / a.nranges), d1 = uniform_i64((r + 1) * a.Nd / a.nranges);
    if (d0 >= d1) return;

    const int Lq = (int)a.Lq, Ld = (int)a.Ld, nb = a.nb;
    const int tiles = (Ld + 31) / 32;  // of a document
    const bool in_lds = a.d_mask && tiles <= kMaskWords;
    const int batch = in_lds ? kMaskWords / tiles : 0x7fffffff;  // documents whose mask LDS holds
    // queries of this unit, tiles of one, passes over the documents if it has more than NTW
    const int i0 = uniform(qb * a.qpw);
    const int nq = uniform((int)(a.Nq - i0 < a.qpw ? a.Nq - i0 : a.qpw));
    const int ntq = a.ntq;

    for (int pass = 0; pass == 0 || pass * NTW < ntq; ++pass) {
        // ---- the unit's query tiles --------------------------------------------
        Token<G> q[NTW];
        uint32_t live = 0;  // bit n: this lane's column of tile n exists and counts
        static_for<0, NTW>([&](auto n) {
            // tile n is tile n % ntq of query n / ntq, or tile pass * NTW + n of the one query
            const int qi = ntq <= NTW ? n / ntq : 0, qt = ntq <= NTW ? n % ntq : pass * NTW + n;
            const bool tile_in = qi < nq && qt < ntq;
            const int64_t i = i0 + (tile_in ? qi : 0);
            const int t0 = tile_in ? qt * 32 : 0, s = t0 + col;
            const int row = s < Lq ? col : Lq - 1 - t0;
            const int64_t tok = i * Lq + t0;
            load_token<G, FAST>(q[n], a.Q + tok * nb * 16, a.q_scale + tok * nb, row, h, nb);
            place_scales<G, FAST>(q[n], h);
            const bool on = tile_in && s < Lq && (!a.q_mask || a.q_mask[i * Lq + s]);
            live |= (uint32_t)on << n;
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

        // Sums of a finished document, tile by tile in order.
        auto finish = [&](int64_t doc) {
            float sum = 0.0f;
            int i = i0, at = 0;  // the query of tile n, and which of its tiles that is
            static_for<0, NTW>([&](auto n) {
                const int tiles_here = ntq <= NTW ? ntq : (ntq - pass * NTW < NTW ? ntq - pass * NTW : NTW);
                if (i < i0 + nq) {
                    float v = m[n];
                    const float o = shfl_xor_f(v, 32);
                    if constexpr (ARGMAX) {
                        const int oi = shfl_xor_i(best[n], 32);
                        const int idx = o > v || (o == v && oi < best[n]) ? oi : best[n];
                        const int s = (ntq <= NTW ? at : pass * NTW + n) * 32 + col;
                        if (h == 0 && s < Lq) a.argmax[(i * a.Nd + doc) * Lq + s] = idx;
                    }
                    v = any && ((live >> n) & 1) ? vmax(v, o) : 0.0f;
                    sum += lanes0_31_sum(v);
                    if (++at == tiles_here) {
                        float* out = a.scores + i * a.Nd + doc;
                        if (lane == 0) *out = pass > 0 ? *out + sum : sum;
                        sum = 0.0f;
                        at = 0;
                        ++i;
                    }
                }
            });
            reset();
            any = false;
        };

        for (int64_t b0 = d0; b0 < d1; b0 += batch) {
            const int64_t b1 = d1 - b0 < batch ? d1 : b0 + batch;
            if (in_lds) {
                const int words = (int)(b1 - b0) * tiles;
                for (int w = lane; w < words; w += 64) {
                    const int64_t doc = b0 + w / tiles;
                    const int t0 = w % tiles * 32;
                    my_mask[w] = mask_word(a.d_mask + doc * Ld + t0, Ld - t0 < 32 ? Ld - t0 : 32);
                }
                lds_fence();
                __builtin_amdgcn_wave_barrier();
            }

            // ---- the stream of tiles ---------------------------------------------
            struct Slot {
                Token<G> t;
                int64_t doc;
                uint32_t bits;
                int tile;
                bool last, valid;
            } slot[P];
            int64_t doc = b0 - 1;  // the tile issued last
            int tile = 0, count = 0;
            uint32_t words = 0;  // this lane's of 64 mask words of doc
            auto issue = [&](Slot& s) {
                ++tile;
                bool valid = true;
                while (tile >= count) {  // the next document with a token
                    if (++doc >= b1) {
                        valid = false;
                        break;
                    }
                    tile = 0;
                    count = tiles;
                    if (in_lds) {
                        count = 0;
                        for (int w0 = 0; w0 < tiles; w0 += 64) {
                            const uint32_t w = w0 + lane < tiles ? my_mask[(int)(doc - b0) * tiles + w0 + lane] : 0;
                            const uint64_t some = __ballot(w != 0);
                            if (some) count = w0 + 64 - __builtin_clzll(some);
                        }
                    }
                    if (count == 0 && pass == 0) {  // nothing to score
                        for (int i = i0; i < i0 + nq; ++i) {
                            if (lane == 0) a.scores[i * a.Nd + doc] = 0.0f;
                            if (ARGMAX)
                                for (int s2 = lane; s2 < Lq; s2 += 64) a.argmax[(i * a.Nd + doc) * Lq + s2] = 0;
                        }
                    }
                }
                s.valid = valid;
                if (!valid) {
                    doc = b1;  // stays behind the end
                    count = 0;
                    tile = 0;
                }
                const int64_t at_doc = valid ? doc : b0;
                const int at_tile = valid ? tile : 0, t0 = at_tile * 32, left = Ld - t0;
                const int64_t tok = at_doc * Ld + t0;
                load_token<G, FAST>(s.t, a.D + tok * nb * 16, a.d_scale + tok * nb, col < left ? col : left - 1, h, nb);
                uint32_t bits = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
                if (in_lds) {
                    if ((at_tile & 63) == 0 && valid)
                        words = at_tile + lane < tiles ? my_mask[(int)(at_doc - b0) * tiles + at_tile + lane] : 0;
                    bits = __builtin_amdgcn_readlane(words, at_tile & 63);
                } else if (a.d_mask && valid) {
                    bits = (uint32_t)__ballot(lane < 32 && lane < left && a.d_mask[at_doc * Ld + t0 + (lane < left ? lane : 0)]);
                }
                s.doc = at_doc;
                s.tile = at_tile;
                s.bits = bits;
                s.last = valid && tile + 1 == count;
            };
            auto consume = [&](Slot& s) {
                place_scales<G, FAST>(s.t, h);
                auto fold = [&](auto masked) {
                    f32x16 start;
#pragma unroll
                    for (int e = 0; e < 16; ++e) start[e] = 0.0f;
                    if constexpr (masked) {
                        const bool on = (s.bits >> col) & 1;
                        const uint32_t mine = s.bits >> (4 * h);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            start[e] = (mine >> (8 * (e >> 2) + (e & 3))) & 1 ? 0.0f : -__builtin_inff();
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            s.t.code[2 * g] = on ? s.t.code[2 * g] : i32x4{};
                            s.t.code[2 * g + 1] = on ? s.t.code[2 * g + 1] : i32x4{};
                            s.t.scale[g] = on ? s.t.scale[g] : 0x7f7f;
                        }
                    }
                    static_for<0, NTW>([&](auto n) {
                        f32x16 acc = start;
                        static_for<0, G>([&](auto g) {
                            acc = mfma32_mx4<0, 0>(s.t.code[2 * g], s.t.scale[g], q[n].code[2 * g], q[n].scale[g], acc);
                            acc = mfma32_mx4<1, 1>(s.t.code[2 * g + 1], s.t.scale[g], q[n].code[2 * g + 1], q[n].scale[g], acc);
                        });
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

            static_for<0, P>([&](auto p) { issue(slot[p]); });
            bool more = slot[0].valid;
            while (more) {
                static_for<0, P>([&](auto p) {
                    if (slot[p].valid) {
                        consume(slot[p]);
                        issue(slot[p]);
                    }
                });
                more = slot[0].valid;
            }
        }
    }
}

// Scores (and argmax) where queries or documents have no tokens.
__global__ __launch_bounds__(256) void zero_mx4_kernel(Mx4FwdArgs a)
{
    const int64_t n = a.Nq * a.Nd, at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t k = at; k < n; k += step) a.scores[k] = 0.0f;
    if (a.argmax)
        for (int64_t k = at; k < n * a.Lq; k += step) a.argmax[k] = 0;
}

int64_t pieces(int64_t n, int b) { return (n + b - 1) / b; }

template <int G, int NTW, int P, bool FAST>
void run(Mx4FwdArgs a, hipStream_t stream)
{
    a.ntq = (int32_t)pieces(a.Lq, 32);
    a.qpw = a.ntq > 0 && a.ntq <= NTW ? NTW / a.ntq : 1;
    a.nqb = (int32_t)pieces(a.Nq, a.qpw);
    // enough units to fill the card's waves twice over, and a range of at least one document
    const int64_t want = pieces((int64_t)device_cu_count() * 32, a.nqb);
    a.nranges = (int32_t)(want < a.Nd ? want : a.Nd);
    const dim3 grid((unsigned)pieces((int64_t)a.nqb * a.nranges, kWaves)), block(kWaves * 64);
    if (a.argmax) hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, true, FAST>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((fwd_mx4_kernel<G, NTW, P, false, FAST>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_fwd_mx4(Mx4FwdArgs a, hipStream_t stream)
{
    if (a.Lq == 0 || a.Ld == 0) {
        const int64_t b = pieces(a.Nq * a.Nd * (a.argmax && a.Lq > 1 ? a.Lq : 1), 256);
        hipLaunchKernelGGL(zero_mx4_kernel, dim3((unsigned)(b < 65536 ? b : 65536)), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    const int G = (a.nb + 3) / 4;
    const bool fast = a.nb % 4 == 0 && (((uintptr_t)a.q_scale | (uintptr_t)a.d_scale) & 3) == 0;
    const int64_t tiles = a.Nq * pieces(a.Lq, 32);
#define MAXSIM_MX4(G, NTW, P) (fast ? run<G, NTW, P, true>(a, stream) : run<G, NTW, P, false>(a, stream))
    if (G == 1) {
        if (tiles <= 1) MAXSIM_MX4(1, 1, 4);
        else if (tiles <= 4) MAXSIM_MX4(1, 4, 4);
        else MAXSIM_MX4(1, 8, 2);
    } else if (G == 2) {
        if (tiles <= 1) run<2, 1, 3, false>(a, stream);
        else run<2, 4, 2, false>(a, stream);
    } else if (G <= 4) {
        run<4, 1, 2, false>(a, stream);
    } else {
        run<8, 1, 1, false>(a, stream);
    }
#undef MAXSIM_MX4
    return hipGetLastError();
}

}  // namespace maxsim
