// Cross-product MaxSim of microscaled 4-bit queries with documents of up to 16 tokens.
//
// A tile of 32 MFMA rows takes 32 / S whole documents in slots of S rows, S the next
// power of two (rows behind a document's last token repeat it): which token a row
// holds is the loading lane's choice, so slots are made of rows whose results land in
// one lane, 16 / S documents in each half of the wave, and the maximum over a
// document is one over S registers. Queries of up to 16 tokens share a tile of
// columns in slots in the same way. The sums over a query's columns take two
// documents at a time, and one store writes those of all documents of the tile. 3
// queries of 5 tokens over 49,824 documents of 8 take 7.7 us (2.6 TB/s; a document a
// tile 28.9), one query over 500,000 documents of 16 110 us (3.8 TB/s; 150). The
// instructions of a tile are the bound: exponents in aligned words were worth 199 to
// 119 us there. Paths of their own for tiles without a masked row made it three times
// the code for 42 queries over 9981 documents of 2 tokens in 14 instead of 16 us.
#include "fwd_mx4.hpp"

namespace maxsim {

namespace {

// Rows of the tile, behind a shift by 4 of the lane's half, that registers
// v S .. v S + S - 1 hold.
template <int LS>
constexpr uint32_t rows_of(int v)
{
    uint32_t rows = 0;
    for (int q = v << LS; q < (v + 1) << LS; ++q) rows |= 1u << (8 * (q >> 2) + (q & 3));
    return rows;
}

template <int G, int NTW, int P, int LS, bool FAST>
__global__ __launch_bounds__(kWaves * 64) void fwd_mx4_short_kernel(Mx4FwdArgs a)
{
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id(), col = lane & 31, h = lane >> 5;
    const int64_t unit = (int64_t)xcd_order(blockIdx.x, gridDim.x) * kWaves + wave;
    if (unit >= (int64_t)a.nqb * a.nranges) return;
    constexpr int S = 1 << LS, NV = 16 / S, per = 2 * NV;  // documents of a half, and of a tile
    const int lq = a.log2_qslot, qpt = 32 >> lq;            // queries of a tile
    const int64_t groups = (a.Nd + per - 1) / per, r = unit / a.nqb;
    const int g0 = uniform((int)(r * groups / a.nranges)), g1 = uniform((int)((r + 1) * groups / a.nranges));
    const int Lq = (int)a.Lq, Ld = (int)a.Ld, nb = a.nb, ntq = a.ntq;
    const int i0 = uniform((int)(unit % a.nqb) * a.qpw);
    const int nq = uniform((int)(a.Nq - i0 < a.qpw ? a.Nq - i0 : a.qpw));

    // the document and the token of the tile's row that this lane loads
    const int reg = (col >> 3) * 4 + (col & 3), in_slot = reg % S;
    const int my_doc = ((col >> 2) & 1) * NV + reg / S, my_tok = in_slot < Ld ? in_slot : Ld - 1;

    for (int q0 = 0; q0 < ntq; q0 += NTW) {  // more than one pass for queries of more than NTW tiles
        const int used = qpt > 1 ? (nq + qpt - 1) / qpt : ntq <= NTW ? nq * ntq : ntq - q0 < NTW ? ntq - q0 : NTW;
        Token<G> q[NTW];
        uint32_t live = 0;  // bit n: this lane's column of tile n exists and counts
        const int64_t base = (int64_t)i0 * Lq + q0 * 32;
        static_for<0, NTW>([&](auto n) __attribute__((always_inline)) {
            const int qi = qpt > 1 ? n * qpt + (col >> lq) : ntq <= NTW ? n / ntq : 0;
            const int s = qpt > 1 ? col & ((1 << lq) - 1) : (ntq <= NTW ? n % ntq : q0 + n) * 32 + col;
            const int row = (qi < nq ? qi : nq - 1) * Lq + (s < Lq ? s : Lq - 1) - q0 * 32;
            load_token<G, FAST, true>(q[n], a.Q + base * nb * 16, a.q_scale + base * nb, row, h, nb);
            place_scales<G, FAST>(q[n], h);
            live |= (uint32_t)(qi < nq && s < Lq && (!a.q_mask || a.q_mask[base + row])) << n;
        });

        struct Slot {
            Token<G> t;
            uint8_t on;
        } slot[P];
        auto issue = [&](Slot& s, int g) __attribute__((always_inline)) {
            const int64_t d0 = (int64_t)g * per;
            const int last = (int)(a.Nd - d0 < per ? a.Nd - d0 : per) - 1;
            const int row = (my_doc < last ? my_doc : last) * Ld + my_tok;
            load_token<G, FAST, false>(s.t, a.D + d0 * Ld * nb * 16, a.d_scale + d0 * Ld * nb, row, h, nb);
            s.on = a.d_mask ? a.d_mask[d0 * Ld + row] : 1;
        };
        auto consume = [&](Slot& s, int g) __attribute__((always_inline)) {
            place_scales<G, FAST>(s.t, h);
            const int64_t d0 = (int64_t)g * per;
            const uint32_t bits = (uint32_t)__ballot(s.on != 0);  // of rows 0 .. 31
            auto put = [&](bool mine, int64_t i, int doc, float sum) __attribute__((always_inline)) {
                if (!mine || d0 + doc >= a.Nd || i >= i0 + nq) return;
                float* out = a.scores + i * a.Nd + d0 + doc;
                *out = q0 > 0 ? *out + sum : sum;
            };
            // Sums over the columns of query i (or of the queries from i on), of the
            // half's NV documents.
            auto flush = [&](float(&sums)[NV], int i) __attribute__((always_inline)) {
                if (qpt == 1) {
                    // the row pairs of two documents are swapped, so that one sum joins both
                    float x[NV > 1 ? NV / 2 : 1];
                    if constexpr (NV == 1) {
                        x[0] = row16_sum(sums[0] + shfl_xor_f(sums[0], 16));
                    } else {
                        static_for<0, NV / 2>([&](auto p) __attribute__((always_inline)) {
                            const auto both = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, sums[2 * p]),
                                                                               __builtin_bit_cast(uint32_t, sums[2 * p + 1]), false, false);
                            x[p] = row16_sum(as_float(both[0]) + as_float(both[1]));
                        });
                    }
                    float sum = x[0];
                    if constexpr (NV > 2)
                        static_for<1, NV / 2>([&](auto p) __attribute__((always_inline)) { sum = (col & 15) == p ? x[p] : sum; });
                    if constexpr (NV == 1) put(col == 0, i, h, sum);
                    else put((col & 15) < NV / 2, i, h * NV + 2 * (col & 15) + (col >> 4), sum);
                } else {
                    static_for<0, NV>([&](auto v) __attribute__((always_inline)) {
                        if (lq > 0) sums[v] = dpp_add<0xB1>(sums[v]);   // quad_perm [1,0,3,2]
                        if (lq > 1) sums[v] = dpp_add<0x4E>(sums[v]);   // quad_perm [2,3,0,1]
                        if (lq > 2) sums[v] = dpp_add<0x141>(sums[v]);  // row_half_mirror
                        if (lq > 3) sums[v] = dpp_add<0x140>(sums[v]);  // row_mirror
                    });
                    for (int v0 = 0; v0 < NV; v0 += 1 << lq) {
                        const int mine = v0 + (col & ((1 << lq) - 1));
                        float sum = sums[0];
                        static_for<1, NV>([&](auto v) __attribute__((always_inline)) { sum = mine == v ? sums[v] : sum; });
                        put(mine < NV, (int64_t)i + (col >> lq), h * NV + mine, sum);
                    }
                }
            };
            f32x16 start;
#pragma unroll
            for (int e = 0; e < 16; ++e) start[e] = 0.0f;
            const uint32_t mine = bits >> (4 * h);
            if (bits != 0xffffffffu) {
                // codes are finite whatever they are; an exponent may be NaN
#pragma unroll
                for (int g = 0; g < G; ++g) s.t.scale[g] = (bits >> col) & 1 ? s.t.scale[g] : 0;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    start[e] = (mine >> (8 * (e >> 2) + (e & 3))) & 1 ? 0.0f : -__builtin_inff();
            }
            float sums[NV];
            static_for<0, NV>([&](auto v) __attribute__((always_inline)) { sums[v] = 0.0f; });
            int i = i0, at = 0;  // the query, and which of its tiles
            static_for<0, NTW>([&](auto n) __attribute__((always_inline)) {
                if (n >= used) return;
                f32x16 acc = start;
                static_for<0, G>([&](auto g) {
                    acc = mfma32_mx4<0, 0>(s.t.code[2 * g], s.t.scale[g], q[n].code[2 * g], q[n].scale[g], acc);
                    acc = mfma32_mx4<1, 1>(s.t.code[2 * g + 1], s.t.scale[g], q[n].code[2 * g + 1], q[n].scale[g], acc);
                });
                stay(acc);
                // what does not count is masked off in bits: no lane branches
                const uint32_t counts = 0u - ((live >> n) & 1);
                static_for<0, NV>([&](auto v) __attribute__((always_inline)) {
                    float m = acc[v * S];
                    static_for<1, S>([&](auto e) __attribute__((always_inline)) { m = vmax(m, acc[v * S + e]); });
                    // (a document without a token that counts scores 0)
                    const uint32_t keep = counts & (0u - (uint32_t)((mine & rows_of<LS>(v)) != 0));
                    sums[v] += as_float(__builtin_bit_cast(uint32_t, m) & keep);
                });
                if (qpt > 1 || ++at == ntq || n + 1 == used) {
                    flush(sums, i);
                    i += qpt;
                    at = 0;
                    static_for<0, NV>([&](auto v) __attribute__((always_inline)) { sums[v] = 0.0f; });
                }
            });
        };

        static_for<0, P>([&](auto p) __attribute__((always_inline)) {
            if (g0 + p < g1) issue(slot[p], g0 + p);
        });
        for (int g = g0; g < g1; g += P) {
            static_for<0, P>([&](auto p) __attribute__((always_inline)) {
                if (g + p >= g1) return;
                consume(slot[p], g + p);
                if (g + p + P < g1) issue(slot[p], g + p + P);
            });
        }
    }
}

// WAVES: units that a CU runs at once.
template <int G, int NTW, int P, int WAVES>
void run_short(Mx4FwdArgs a, hipStream_t stream)
{
    const int64_t per = 32 >> a.log2_slot, groups = (a.Nd + per - 1) / per;
    a.qpw = a.ntq > NTW ? 1 : NTW / a.ntq * (32 >> a.log2_qslot);
    a.nqb = (int32_t)pieces(a.Nq, a.qpw);
    const int64_t units = (int64_t)device_cu_count() * WAVES, want = units / a.nqb > 0 ? units / a.nqb : 1;
    a.nranges = (int32_t)(want < groups ? want : groups);
    const dim3 grid((unsigned)pieces((int64_t)a.nqb * a.nranges, kWaves)), block(kWaves * 64);
    const bool fast = fast_rows<G>(a);
    auto launch = [&](auto log2_slot) {
        constexpr int LS = log2_slot;
        if constexpr (G == 1) {  // (wider tokens: little of their time)
            if (fast) {
                hipLaunchKernelGGL((fwd_mx4_short_kernel<G, NTW, P, LS, true>), grid, block, 0, stream, a);
                return;
            }
        }
        hipLaunchKernelGGL((fwd_mx4_short_kernel<G, NTW, P, LS, false>), grid, block, 0, stream, a);
    };
    if (a.log2_slot == 4) launch(std::integral_constant<int, 4>{});
    else if (a.log2_slot == 3) launch(std::integral_constant<int, 3>{});
    else if (a.log2_slot == 2) launch(std::integral_constant<int, 2>{});
    else if (a.log2_slot == 1) launch(std::integral_constant<int, 1>{});
    else launch(std::integral_constant<int, 0>{});
}

}  // namespace

// 42 queries of 64 tokens over 9981 documents of 2 tokens take 15.4 us, 97 with a document
// a tile; one query over 500,000 documents of 16 110 and 150. Where there is less than
// a tile for each CU, a document a tile spreads further (10 queries of 48 tokens, 56
// documents of one, 1024 channels: 9.3 us against 13.1), so this is refused (false).
bool launch_fwd_mx4_short(Mx4FwdArgs a, hipStream_t stream)
{
    if (a.Ld > 16 || a.argmax) return false;
    a.log2_slot = log2_up(a.Ld);
    a.log2_qslot = a.Lq <= 16 ? log2_up(a.Lq) : 5;
    const int64_t groups = pieces(a.Nd, 32 >> a.log2_slot);
    const int64_t tiles = a.ntq > 1 ? a.Nq * a.ntq : pieces(a.Nq, 32 >> a.log2_qslot);
    if (tiles * groups < device_cu_count()) return false;
    const bool many = tiles > 1 && tiles * groups >= 16 * (int64_t)device_cu_count();
    if (a.nb <= 4) {
        if (many) run_short<1, 4, 2, 8>(a, stream);
        else run_short<1, 1, 4, 16>(a, stream);
    } else if (a.nb <= 8) {
        if (many) run_short<2, 4, 2, 8>(a, stream);
        else run_short<2, 1, 2, 8>(a, stream);
    } else if (a.nb <= 16) {
        run_short<4, 1, 2, 8>(a, stream);
    } else {
        run_short<8, 1, 1, 8>(a, stream);
    }
    return true;
}

}  // namespace maxsim
