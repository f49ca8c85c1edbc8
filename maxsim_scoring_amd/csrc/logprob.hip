// Log probabilities of given columns under the softmax of their row of scores,
// with ranks, entropy and the row's best columns, and their gradient, for gfx950.
//
// Forward. A row is cut into chunks of 4096 columns, one workgroup each, 16 columns
// a thread in registers, read once: the largest score, the sums of exp(z) and of
// exp(z) z against it, how many columns come before each target, and the candidates
// for the best columns. Rows of one chunk finish there (those of up to 256 or 512
// columns in one wave); otherwise a second launch joins the chunks of a row. Few long
// rows spread over the card in this way.
//
// 128 rows of 128 columns, one target, 8 best: 5.2 us. 32 rows of 100,000, 8 targets,
// 100 best: 14.3 us, and 8.2 us the join of 25 chunks a row. Not the 12.8 MB of
// scores (2.4 us at a copy's rate) but instructions are the bound: of 14,500 cycles of
// a workgroup 4,700 count ranks (two instructions for each score and target), 4,900
// select and copy the best, and 2,000 wait for the scores.
//
// The sums take 2^t with t = (x - m) scale log2(e) from the hardware, off by 4 units
// of 2^-24 |z| for the three roundings of t; they are float64, so that a row whose
// largest probability is close to 1 keeps its entropy.
//
// Best columns. Scores map to 32-bit keys in float order. A histogram of 256 equal
// bins between the chunk's least and largest key finds the bin of the k-th: first of
// the threads' largest keys alone, which seldom leaves many more than k, otherwise of
// all keys (32 x 100,000 as above: 23.8 us with all keys only, 22.5 us so); it is cut
// into 256 again only while more than k + k/2 + 32 lie at or above its lower edge.
// Equal keys that are too many are told apart by their columns in the same way. What
// is left is ordered by counting, for each, how many are larger.
//
// Backward. One pass, element-wise but for the targets: their gradients are added
// into a chunk of columns in LDS by one wave, in the order of the targets. 512 rows of
// 100,000 columns with 32 targets and the entropy's gradient: 410 MB in 79 us, 5.2
// TB/s; 128 rows of 128 columns: 3.5 us.
#include "logprob.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

constexpr int kBins = 256;
constexpr int kMaxCap = 2048;     // logprob_cap(1024) and more, a power of two
constexpr int kJoinThreads = 512;
constexpr int kJoinHeld = 16;     // candidates that a thread of the join holds

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));

template <int E> constexpr int elem_bytes() { return E == kF32 ? 4 : 2; }

// Keys in float order, -0 as +0. (A NaN may have any key: a row that holds one is
// marked by its largest score.)
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t k)
{
    return __builtin_bit_cast(float, (k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// exp(z) for z <= 0 (0 below -200); NaN for NaN.
__device__ __forceinline__ float exp_neg(float z)
{
    constexpr float kHi = 0x1.715476p0f, kLo = 0x1.4ae0c0p-26f;  // log2(e)
    const float t = z * kHi;
    const float rest = __builtin_fmaf(z, kHi, -t) + z * kLo;
    // the hardware's 2^x gives no subnormals: small ones are made 2^64 larger first
    const bool small = t < -100.0f;
    const float e = __builtin_amdgcn_exp2f(small ? t + 64.0f : t);
    return __builtin_fmaf(e * 0x1.62e430p-1f, rest, e) * (small ? 0x1p-64f : 1.0f);  // e (1 + rest log 2)
}
// 1 - exp(-z) for z in [0, 1/2): the series, whose next term is below 2^-26 of the sum.
__device__ __forceinline__ float one_minus_exp(float z)
{
    float s = 1.0f / 40320.0f;
    constexpr float c[7] = {1.0f / 5040.0f, 1.0f / 720.0f, 1.0f / 120.0f, 1.0f / 24.0f, 1.0f / 6.0f, 0.5f, 1.0f};
#pragma unroll
    for (int k = 0; k < 7; ++k) s = __builtin_fmaf(-z, s, c[k]);
    return z * s;
}
__device__ __forceinline__ float floor_z(float z) { return z < -200.0f ? -200.0f : z; }

// A row's columns c0 + place, N per thread of T: value v of a thread is column
// place(v) of the chunk; V consecutive ones come in one load.
template <int E, int T, int N>
struct Layout {
    static constexpr int V = E == kF32 ? 4 : 8;
    static constexpr int kColumns = T * N;
    __device__ static __forceinline__ int place(int v) { return ((v / V) * T + (int)threadIdx.x) * V + v % V; }
};

// The thread's columns of row i from c0 on: NaN-free loading of what exists and is
// not masked, -Inf elsewhere.
template <int E, int T, int N>
__device__ __forceinline__ void load_columns(const LogprobArgs& a, int64_t i, int c0, float (&x)[N])
{
    typedef Layout<E, T, N> Y;
    const int n = a.Nd - c0 < Y::kColumns ? a.Nd - c0 : Y::kColumns;
    const char* p = (const char*)a.X + (i * a.Nd + c0) * elem_bytes<E>();
    const uint8_t* mp = a.mask ? a.mask + i * a.Nd + c0 : nullptr;
#pragma unroll
    for (int g = 0; g < N / Y::V; ++g) {
        const int at = Y::place(g * Y::V);
        u32x4 w;
        if (at + Y::V <= n) {
            w = *(const u32x4_any*)(p + (int64_t)at * elem_bytes<E>());
        } else {
            // -Inf behind the end: 0xff800000, 0xff80 or 0xfc00
            constexpr uint32_t kNone = E == kF32 ? 0xff800000u : E == kBF16 ? 0xff80ff80u : 0xfc00fc00u;
            w = u32x4{kNone, kNone, kNone, kNone};
#pragma unroll
            for (int e = 0; e < Y::V; ++e) {
                if (at + e >= n) continue;
                if constexpr (E == kF32) w[e] = ((const uint32_t*)p)[at + e];
                else {
                    const uint32_t b = ((const uint16_t*)p)[at + e];
                    w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | b << 16 : (w[e / 2] & 0xffff0000u) | b;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < Y::V; ++e) {
            if constexpr (E == kF32) x[g * Y::V + e] = as_float(w[e]);
            else {
                const uint32_t bits = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
                x[g * Y::V + e] = E == kBF16 ? as_float(bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
            }
        }
    }
    if (!mp) return;
#pragma unroll
    for (int g = 0; g < N / Y::V; ++g) {
        const int at = Y::place(g * Y::V);
        uint32_t keep[Y::V / 4];
#pragma unroll
        for (int k = 0; k < Y::V / 4; ++k) {
            keep[k] = 0;
            if (at + Y::V <= n) keep[k] = *(const u32_any*)(mp + at + 4 * k);
            else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (at + 4 * k + e < n) keep[k] |= (uint32_t)mp[at + 4 * k + e] << (8 * e);
            }
        }
#pragma unroll
        for (int e = 0; e < Y::V; ++e)
            x[g * Y::V + e] = (keep[e / 4] >> (8 * (e & 3))) & 0xffu ? x[g * Y::V + e] : -__builtin_inff();
    }
}

template <int E>
__device__ __forceinline__ float load_one(const LogprobArgs& a, int64_t i, int c)
{
    if (a.mask && !a.mask[i * a.Nd + c]) return -__builtin_inff();
    if constexpr (E == kF32) return ((const float*)a.X)[i * a.Nd + c];
    else {
        const uint16_t b = ((const uint16_t*)a.X)[i * a.Nd + c];
        return E == kBF16 ? __builtin_bit_cast(float, (uint32_t)b << 16) : (float)__builtin_bit_cast(_Float16, b);
    }
}

// Reductions over a wave, the same result in every lane: rows of 16 lanes by DPP,
// the four rows through scalar registers.
template <int CTRL, typename V>
__device__ __forceinline__ V dpp_of(V v)
{
    if constexpr (sizeof(V) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, false);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
    }
}
template <typename V>
__device__ __forceinline__ V lane_of(V v, int lane)
{
    if constexpr (sizeof(V) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    }
}
template <typename V, typename OP>
__device__ __forceinline__ V wave_reduce(V v, OP op)
{
    v = op(v, dpp_of<0xB1>(v));   // quad_perm [1,0,3,2]
    v = op(v, dpp_of<0x4E>(v));   // quad_perm [2,3,0,1]
    v = op(v, dpp_of<0x141>(v));  // row_half_mirror
    v = op(v, dpp_of<0x140>(v));  // row_mirror
    return op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
}
struct AddOp { template <typename V> __device__ __forceinline__ V operator()(V a, V b) const { return a + b; } };
struct MinOp { __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; } };
// the maximum that is NaN where either is
struct MaxOp { __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_elementwise_maximum(a, b); } };

// Sums of lanes 0 .. l: within rows of 16 lanes by row_shr, then the last lane of
// each row (of each half) to the next.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v)
{
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);  // row_bcast:15
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);  // row_bcast:31
    return v;
}

// The waves' results joined in order; put by one lane of each wave, a barrier between.
template <int W, typename V>
__device__ __forceinline__ void put(V (&red)[W], V v)
{
    if (W > 1 && lane_id() == 0) red[threadIdx.x >> 6] = v;
}
template <int W, typename V, typename OP>
__device__ __forceinline__ V joined(const V (&red)[W], V v, OP op)
{
    if constexpr (W > 1) {
        v = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = op(v, red[w]);
    }
    return v;
}

// Order of the output as a number: the key, then the lower column first. All of a
// row's are different.
__device__ __forceinline__ uint64_t order_of(uint32_t key, int col, int cbits)
{
    return (uint64_t)key << cbits | (uint64_t)(((uint32_t)1 << cbits) - 1u - (uint32_t)col);
}
__device__ __forceinline__ int column_of(uint64_t o, int cbits)
{
    const uint32_t m = ((uint32_t)1 << cbits) - 1u;
    return (int)(m - ((uint32_t)o & m));
}

// A bound of a set of numbers between lo and hi such that at least K of them, with
// `above` others beyond hi, are at or above it; upto becomes how many. That is at
// most cap, or the bound is the K-th largest itself. each(f) calls f(number) for
// each of this thread's. hist: LDS of kBins + 3.
template <int T, typename U, typename Each>
__device__ __forceinline__ U select_bound(Each each, uint32_t K, uint32_t cap, U lo, U hi, uint32_t& above, uint32_t& upto,
                                          uint32_t* hist)
{
    int shift = 64 - __builtin_clzll((uint64_t)(hi - lo) | 1) - 8;  // 256 bins of 2^shift cover them
    if (shift < 0) shift = 0;
    U bins = kBins;
    for (;;) {
        for (int k = threadIdx.x; k < kBins; k += T) hist[k] = 0;
        __syncthreads();
        each([&](U o) {
            const U bin = (U)(o - lo) >> shift;
            if (o >= lo && bin < bins) atomicAdd(&hist[(uint32_t)bin], 1u);
        });
        __syncthreads();
        if (threadIdx.x < 64) {
            // lane 0 holds the top bins; the bin where the count from the top reaches K
            const int lane = threadIdx.x;
            uint32_t c[4], mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) mine += c[e] = hist[255 - (4 * lane + e)];
            uint32_t before = above + wave_scan(mine) - mine;
            uint32_t bin = 0, over = 0, up = 0;
            bool found = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (before < K && K <= before + c[e]) {
                    bin = (uint32_t)(255 - (4 * lane + e));
                    over = before;
                    up = before + c[e];
                    found = true;
                }
                before += c[e];
            }
            if (found) {  // one lane
                hist[kBins] = bin;
                hist[kBins + 1] = over;
                hist[kBins + 2] = up;
            }
        }
        __syncthreads();
        lo += (U)hist[kBins] << shift;
        above = hist[kBins + 1];
        upto = hist[kBins + 2];
        if (upto <= cap || shift == 0) return lo;
        bins = shift < 8 ? (U)1 << shift : (U)kBins;  // the bin and nothing beyond it
        shift = shift > 8 ? shift - 8 : 0;
    }
}

// What the best columns are picked from, value by value (for_all calls f(v) as often
// in every lane): N scores of a thread's columns, N numbers in registers, or numbers in
// memory. above: is value v a candidate whose key is at least the bound's?
struct Bound {
    uint32_t key;
    float x;          // its score
    uint64_t number;  // the least with that key
};
template <int E, int T, int N>
struct Scores {
    const float (&x)[N];
    int c0, cbits;
    template <typename F> __device__ __forceinline__ void for_all(F f) const { static_for<0, N>(f); }
    __device__ __forceinline__ bool is(int v) const { return x[v] > -__builtin_inff(); }
    __device__ __forceinline__ uint32_t key(int v) const { return key_of(x[v]); }
    __device__ __forceinline__ uint64_t number(int v) const { return order_of(key(v), c0 + Layout<E, T, N>::place(v), cbits); }
    __device__ __forceinline__ bool above(int v, const Bound& b) const { return x[v] >= b.x; }
};
template <int N>
struct Numbers {
    const uint64_t (&o)[N];
    int cbits;
    template <typename F> __device__ __forceinline__ void for_all(F f) const { static_for<0, N>(f); }
    __device__ __forceinline__ bool is(int v) const { return o[v] != 0; }
    __device__ __forceinline__ uint32_t key(int v) const { return (uint32_t)(o[v] >> cbits); }
    __device__ __forceinline__ uint64_t number(int v) const { return o[v]; }
    __device__ __forceinline__ bool above(int v, const Bound& b) const { return o[v] >= b.number; }
};
struct Far {
    const uint64_t* o;
    int n, stride, cbits;
    template <typename F> __device__ __forceinline__ void for_all(F f) const
    {
        for (int v = 0; v * stride < n; ++v) f(v);
    }
    __device__ __forceinline__ uint64_t number(int v) const
    {
        const int e = v * stride + (int)threadIdx.x;
        return e < n ? o[e] : 0;
    }
    __device__ __forceinline__ bool is(int v) const { return number(v) != 0; }
    __device__ __forceinline__ uint32_t key(int v) const { return (uint32_t)(number(v) >> cbits); }
    __device__ __forceinline__ bool above(int v, const Bound& b) const { return number(v) >= b.number; }
};

// Picks the best columns into to[0, n), n <= cap, in any order. least, top: the range
// of the candidates' keys; have: how many there are in all; threads: how many of the
// workgroup's hold one; best: this thread's largest key (0: it holds none). counter: 0.
//
// A bound that K threads' largest keys reach has K candidates at or above it, and for
// K up to half of the threads seldom many more; it takes one number of each thread.
// Only where they are too many are all candidates looked at.
template <int T, typename Source>
__device__ __forceinline__ uint32_t pick(const Source& from, int have, int threads, uint32_t best, uint32_t least, uint32_t top,
                                         const LogprobArgs& a, uint64_t* to, uint32_t* hist, uint32_t* counter)
{
    const uint32_t K = (uint32_t)a.K, cap = (uint32_t)a.cap;
    // a wave takes a run of places; which one depends on the waves' timing, the
    // outputs do not: they are ordered later
    auto copy = [&](auto taken) {
        uint32_t mine = 0;
        from.for_all([&](int v) { mine += (uint32_t)__builtin_popcountll(__ballot(taken(v))); });
        if (mine != 0) {
            uint32_t at = 0;
            if (lane_id() == 0) at = atomicAdd(counter, mine);
            at = (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
            from.for_all([&](int v) {
                const bool t = taken(v);
                const uint64_t all = __ballot(t);
                if (all == 0) return;
                const uint32_t place = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
                if (t && place < cap) to[place] = from.number(v);
                at += (uint32_t)__builtin_popcountll(all);
            });
        }
        __syncthreads();
        return *counter;
    };
    auto copy_from = [&](uint32_t key) {
        const Bound b = {key, score_of(key), (uint64_t)key << a.cbits};
        return copy([&](int v) { return from.above(v, b); });
    };
    uint32_t key = least, above = 0, upto = (uint32_t)have;
    if (upto > cap && 2 * K <= (uint32_t)T && K <= (uint32_t)threads) {
        // (as many may be above it as there are threads: one round of bins is enough)
        key = select_bound<T, uint32_t>(
            [&](auto f) {
                if (best != 0) f(best);
            },
            K, (uint32_t)T, least, top, above, upto, hist);
        const uint32_t n = copy_from(key);
        if (n <= cap) return n;
        least = key;
        above = 0;
        upto = n;
        __syncthreads();  // the counter is read
        if (threadIdx.x == 0) *counter = 0;
    }
    if (upto <= cap) return copy_from(key);
    key = select_bound<T, uint32_t>(
        [&](auto f) {
            from.for_all([&](int v) {
                if (from.is(v)) f(from.key(v));
            });
        },
        K, cap, least, top, above, upto, hist);
    if (upto <= cap) return copy_from(key);
    // equal keys are told apart by their columns
    const uint64_t border = select_bound<T, uint64_t>(
        [&](auto f) {
            from.for_all([&](int v) {
                if (from.is(v) && from.key(v) == key) f(from.number(v));
            });
        },
        K, cap, order_of(key, a.Nd - 1, a.cbits), order_of(key, 0, a.cbits), above, upto, hist);
    const uint32_t n = copy([&](int v) { return from.is(v) && from.number(v) >= border; });
    return n < cap ? n : cap;
}

// In float64, where neither the difference of two scores nor its product overflows.
__device__ __forceinline__ float logp_of(const LogprobArgs& a, float x, float m, double L)
{
    return (float)((double)a.scale * ((double)x - (double)m) - L);
}

// Writes the K best of n <= kMaxCap numbers of cand (LDS) in order.
template <int T>
__device__ __forceinline__ void write_best(const LogprobArgs& a, int64_t i, const uint64_t* cand, int n, float m, double L)
{
    for (int e = threadIdx.x; e < n; e += T) {
        const uint64_t mine = cand[e];
        int place = 0;
#pragma unroll 8
        for (int k = 0; k < n; ++k) place += cand[k] > mine;
        if (place < a.K) {
            const float x = score_of((uint32_t)(mine >> a.cbits));
            a.top_idx[i * a.K + place] = column_of(mine, a.cbits);
            a.top_logp[i * a.K + place] = logp_of(a, x, m, L);
        }
    }
    for (int e = n + threadIdx.x; e < a.K; e += T) {
        a.top_idx[i * a.K + e] = -1;
        a.top_logp[i * a.K + e] = L == L ? -__builtin_inff() : (float)L;
    }
}

// A row's statistics. A NaN or +Inf among the candidates makes the sum NaN, and
// with it every float output of the row.
__device__ __forceinline__ double sum_of(float m, double sum)
{
    return m < __builtin_inff() ? sum : __builtin_nan("");
}
__device__ __forceinline__ void write_stats(const LogprobArgs& a, int64_t i, float m, double sum, double sum_t, double L)
{
    a.norm[2 * i] = L == L ? m : __builtin_nanf("");
    a.norm[2 * i + 1] = (float)L;
    if (a.entropy) a.entropy[i] = sum == 0.0 ? 0.0f : (float)(L - sum_t * 0x1.62e42fefa39efp-1 / sum);  // z = t log 2
}

// Target p of a row: column c (-1: none named) with score x (-Inf: no candidate),
// `before` candidates before it.
__device__ __forceinline__ void write_target(const LogprobArgs& a, int64_t i, int p, int c, float x, uint32_t before, float m, double L)
{
    const bool in = x != -__builtin_inff();
    float lp = c >= 0 ? x : 0.0f;
    if (in || L != L) lp = logp_of(a, x, m, L);
    a.logp[i * a.P + p] = lp;
    if (a.rank) a.rank[i * a.P + p] = in ? (int)before : -1;
}

template <int E>
__device__ __forceinline__ int target_of(const LogprobArgs& a, int64_t i, int p, float& x)
{
    int c = p < a.P ? a.targets[i * a.P + p] : -1;
    if (c >= a.Nd || c < 0) c = -1;
    x = c >= 0 ? load_one<E>(a, i, c) : -__builtin_inff();
    return c;
}

// The largest float below x (-Inf below the lowest); NaN for NaN.
__device__ __forceinline__ float float_below(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    if (x != x) return x;
    if (x == 0.0f) return -0x1p-149f;
    return as_float(x > 0.0f ? b - 1 : b + 1);
}

// 2^t of scores against the largest, t at least -200 (where 2^t is 0): so for -Inf,
// and in rows without candidates.
__device__ __forceinline__ float t_of(float x, float m, float c) { return __builtin_fmaxf((x - m) * c, -200.0f); }

// One chunk of a row, N columns a thread. WHOLE: the row's only one.
template <int E, int T, int N, bool WHOLE>
__global__ __launch_bounds__(T) void logprob_part_kernel(LogprobArgs a)
{
    typedef Layout<E, T, N> Y;
    constexpr int W = T / 64;
    __shared__ uint32_t hist[kBins + 4];
    __shared__ uint64_t cand[kMaxCap];
    __shared__ float red_m[W];
    __shared__ uint32_t red_least[W], red_have[W], red_threads[W], counter;
    __shared__ double red_sum[W], red_t[W];
    __shared__ uint32_t counts[W][64];

    const int64_t unit = blockIdx.x, i = WHOLE ? unit : unit / a.chunks;
    const int c0 = WHOLE ? 0 : (int)(unit % a.chunks) * Y::kColumns;
    const int wave = threadIdx.x >> 6, lane = lane_id();
    if (threadIdx.x == 0) counter = 0;
    float x[N];
    load_columns<E, T, N>(a, i, c0, x);
    float tx;  // target `lane`
    int tc = target_of<E>(a, i, lane, tx);

    float m = x[0];
    uint32_t least = 0xffffffffu, have = 0, threads = 0, best = 0;
#pragma unroll
    for (int v = 1; v < N; ++v) m = MaxOp{}(m, x[v]);
    if (m > -__builtin_inff()) best = key_of(m);
    m = wave_reduce(m, MaxOp{});
    put(red_m, m);
    if (a.K) {
        float low = __builtin_inff();
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const bool in = x[v] > -__builtin_inff();
            have += (uint32_t)__builtin_popcountll(__ballot(in));
            low = in && x[v] < low ? x[v] : low;
        }
        least = key_of(low);
        least = wave_reduce(least, MinOp{});
        threads = (uint32_t)__builtin_popcountll(__ballot(best != 0));
        put(red_least, least);
        put(red_have, have);
        put(red_threads, threads);
    }
    if (W > 1) __syncthreads();
    m = joined(red_m, m, MaxOp{});

    const float scale2 = a.scale * 0x1.715476p0f;  // log2(e)
    double sum = 0.0, sum_t = 0.0;
#pragma unroll
    for (int v = 0; v < N; ++v) {
        const float t = t_of(x[v], m, scale2), e = __builtin_amdgcn_exp2f(t);
        sum += (double)e;
        sum_t = __builtin_fma((double)e, (double)t, sum_t);
    }
    sum = wave_reduce(sum, AddOp{});
    sum_t = wave_reduce(sum_t, AddOp{});
    put(red_sum, sum);
    put(red_t, sum_t);

    // ---- how many come before each target, 64 targets at a time --------------
    // Equal scores come before the target if their column does: none of a chunk behind
    // it, all of one in front of it. x >= xt is x > the float below xt. Four targets at
    // a time, two in the halves of a word when they are added up over the wave. (A
    // ballot and a bit count for each register instead wait for each other.)
    auto count_before = [&](int p0) {  // that of target p0 + lane
        const int np = a.P - p0 < 64 ? a.P - p0 : 64;
        uint32_t mine = 0;
        auto some = [&](auto width, int p) {
            constexpr int M = width;
            float xt[M], least[M];
            int t[M];
            bool here = false;
#pragma unroll
            for (int k = 0; k < M; ++k) {
                xt[k] = lane_of(tx, p + k);
                t[k] = lane_of(tc, p + k) - c0;
                here |= t[k] >= 0 && t[k] < Y::kColumns;
                least[k] = t[k] < 0 ? xt[k] : float_below(xt[k]);
            }
            uint32_t n[M] = {};
            if (here) {
#pragma unroll
                for (int v = 0; v < N; ++v)
#pragma unroll
                    for (int k = 0; k < M; ++k) n[k] += x[v] > (Y::place(v) < t[k] ? least[k] : xt[k]);
            } else {
#pragma unroll
                for (int v = 0; v < N; ++v)
#pragma unroll
                    for (int k = 0; k < M; ++k) n[k] += x[v] > least[k];
            }
            if constexpr (M == 1) {
                const uint32_t all = wave_reduce(n[0], AddOp{});
                mine = lane == p ? all : mine;
            } else {
#pragma unroll
                for (int k = 0; k < M; k += 2) {
                    const uint32_t both = wave_reduce(n[k] | n[k + 1] << 16, AddOp{});
                    mine = lane == p + k ? both & 0xffffu : lane == p + k + 1 ? both >> 16 : mine;
                }
            }
        };
        int p = 0;
        for (; p + 4 <= np; p += 4) some(std::integral_constant<int, 4>{}, p);
        for (; p < np; ++p) some(std::integral_constant<int, 1>{}, p);
        counts[wave][lane] = mine;
    };
    auto counted = [&] {
        uint32_t n = counts[0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) n += counts[w][lane];
        return n;
    };

    double L = 0.0;
    for (int p0 = 0; p0 == 0 || p0 < a.P; p0 += 64) {
        if (p0 > 0) tc = target_of<E>(a, i, p0 + lane, tx);
        if (a.rank) count_before(p0);
        __syncthreads();  // counts, and the sums in the first round
        if (p0 == 0) {
            sum = sum_of(m, joined(red_sum, sum, AddOp{}));
            sum_t = joined(red_t, sum_t, AddOp{});
            if constexpr (WHOLE) {
                L = log(sum);
                if (threadIdx.x == 0) write_stats(a, i, m, sum, sum_t, L);
            } else if (threadIdx.x == 0) {
                a.ws_top[unit] = m;
                a.ws_sums[2 * unit] = sum;
                a.ws_sums[2 * unit + 1] = sum_t;
            }
        }
        if (wave == 0 && p0 + lane < a.P) {
            if constexpr (WHOLE) write_target(a, i, p0 + lane, tc, tx, a.rank ? counted() : 0, m, L);
            else if (a.rank) a.ws_rank[unit * a.P + p0 + lane] = counted();
        }
        if (p0 + 64 < a.P) __syncthreads();  // counts are read
    }
    if (a.K == 0) return;

    // ---- candidates for the best columns --------------------------------------
    have = joined(red_have, have, AddOp{});
    least = joined(red_least, least, MinOp{});
    threads = joined(red_threads, threads, AddOp{});
    const uint32_t n = pick<T>(Scores<E, T, N>{x, c0, a.cbits}, (int)have, (int)threads, best, least, key_of(m), a, cand, hist, &counter);
    if constexpr (WHOLE) {
        write_best<T>(a, i, cand, (int)n, m, L);
    } else {
        // every chunk leaves cap numbers, so that the join reads them without counts
        for (int e = threadIdx.x; e < a.cap; e += T) a.ws_cand[unit * a.cap + e] = e < (int)n ? cand[e] : 0;
    }
}

// Joins the chunks of a row.
template <int E>
__global__ __launch_bounds__(kJoinThreads) void logprob_join_kernel(LogprobArgs a)
{
    constexpr int T = kJoinThreads, W = T / 64;
    __shared__ uint32_t hist[kBins + 4];
    __shared__ uint64_t cand[kMaxCap];
    __shared__ float red_m[W];
    __shared__ uint32_t red_least[W], red_have[W], red_threads[W], counter;
    __shared__ double red_sum[W], red_t[W];

    if (threadIdx.x == 0) counter = 0;
    const int64_t i = blockIdx.x, u0 = i * a.chunks;
    const int total = a.K ? a.chunks * a.cap : 0;  // candidates, 0 where a chunk had fewer
    const bool in_registers = total <= T * kJoinHeld;
    const uint64_t* from = a.ws_cand + u0 * a.cap;
    // What the row's outputs need is loaded at once: every dependent load would add
    // a memory latency to the few workgroups' time.
    const int tid = threadIdx.x;
    float tx, first_top = -__builtin_inff();
    double first_sum = 0.0, first_t = 0.0;
    int tc = target_of<E>(a, i, tid, tx);
    if (tid < a.chunks) {
        first_top = a.ws_top[u0 + tid];
        first_sum = a.ws_sums[2 * (u0 + tid)];
        first_t = a.ws_sums[2 * (u0 + tid) + 1];
    }
    auto count_of = [&](int p) {
        uint32_t n = 0;
#pragma unroll 8
        for (int c = 0; c < a.chunks; ++c) n += a.ws_rank[(u0 + c) * a.P + p];
        return n;
    };
    uint32_t before = a.rank && tid < a.P ? count_of(tid) : 0;
    uint64_t o[kJoinHeld];
    uint32_t least = 0xffffffffu, have = 0, best = 0;
    for (int e0 = 0; e0 < total; e0 += kJoinHeld * T) {
#pragma unroll
        for (int k = 0; k < kJoinHeld; ++k) {
            const int e = e0 + k * T + (int)threadIdx.x;
            o[k] = e < total ? from[e] : 0;
        }
#pragma unroll
        for (int k = 0; k < kJoinHeld; ++k) {
            const uint32_t key = (uint32_t)(o[k] >> a.cbits);  // 0 of none
            have += o[k] != 0;
            least = o[k] != 0 ? MinOp{}(least, key) : least;
            best = key > best ? key : best;
        }
    }
    float m = first_top;
    for (int c = tid + T; c < a.chunks; c += T) m = MaxOp{}(m, a.ws_top[u0 + c]);
    m = wave_reduce(m, MaxOp{});
    put(red_m, m);
    least = wave_reduce(least, MinOp{});
    put(red_least, least);
    have = wave_reduce(have, AddOp{});
    put(red_have, have);
    uint32_t threads = (uint32_t)__builtin_popcountll(__ballot(best != 0));
    put(red_threads, threads);
    __syncthreads();
    m = joined(red_m, m, MaxOp{});

    const float scale2 = a.scale * 0x1.715476p0f;
    double sum = 0.0, sum_t = 0.0;
    auto add = [&](float top, double s, double st) {
        const float t = t_of(top, m, scale2);
        const double e = (double)__builtin_amdgcn_exp2f(t);
        sum = __builtin_fma(e, s, sum);
        sum_t = __builtin_fma(e, __builtin_fma((double)t, s, st), sum_t);
    };
    if (tid < a.chunks) add(first_top, first_sum, first_t);
    for (int c = tid + T; c < a.chunks; c += T) add(a.ws_top[u0 + c], a.ws_sums[2 * (u0 + c)], a.ws_sums[2 * (u0 + c) + 1]);
    sum = wave_reduce(sum, AddOp{});
    sum_t = wave_reduce(sum_t, AddOp{});
    put(red_sum, sum);
    put(red_t, sum_t);
    __syncthreads();
    sum = sum_of(m, joined(red_sum, sum, AddOp{}));
    sum_t = joined(red_t, sum_t, AddOp{});
    const double L = log(sum);
    if (threadIdx.x == 0) write_stats(a, i, m, sum, sum_t, L);
    for (int p = tid; p < a.P; p += T) {
        if (p >= T) {
            tc = target_of<E>(a, i, p, tx);
            before = a.rank ? count_of(p) : 0;
        }
        write_target(a, i, p, tc, tx, before, m, L);
    }
    if (a.K == 0) return;

    have = joined(red_have, have, AddOp{});
    least = joined(red_least, least, MinOp{});
    threads = joined(red_threads, threads, AddOp{});
    const uint32_t n = in_registers
        ? pick<T>(Numbers<kJoinHeld>{o, a.cbits}, (int)have, (int)threads, best, least, key_of(m), a, cand, hist, &counter)
        : pick<T>(Far{from, total, T, a.cbits}, (int)have, (int)threads, best, least, key_of(m), a, cand, hist, &counter);
    write_best<T>(a, i, cand, (int)n, m, L);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

template <int OUT, int V>
__device__ __forceinline__ void store_columns(void* dX, int64_t at, int n, const float* y)
{
    if (n >= V) {
        if constexpr (OUT == kF32) {
            float* p = (float*)dX + at;
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                u32x4 w;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __builtin_bit_cast(uint32_t, y[e + k]);
                *(u32x4_any*)(p + e) = w;
            }
        } else {
            uint16_t* p = (uint16_t*)dX + at;
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
                *(u32x2_any*)(p + e) = u32x2{half_pair<OUT>(y[e], y[e + 1]), half_pair<OUT>(y[e + 2], y[e + 3])};
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (e >= n) continue;
        if constexpr (OUT == kF32) ((float*)dX)[at + e] = y[e];
        else ((uint16_t*)dX)[at + e] = (uint16_t)half_bits(OUT, y[e]);
    }
}

template <int E, int T, int N>
__global__ __launch_bounds__(T) void logprob_bwd_kernel(LogprobArgs a)
{
    typedef Layout<E, T, N> Y;
    __shared__ float add[Y::kColumns];  // the targets' gradients, by column
    __shared__ int cols[T];
    __shared__ float grads[T];
    __shared__ float red[2][T / 64];

    const int64_t unit = blockIdx.x, i = unit / a.chunks;
    const int c0 = (int)(unit % a.chunks) * Y::kColumns;
    float x[N];
    load_columns<E, T, N>(a, i, c0, x);
    for (int k = threadIdx.x; k < Y::kColumns; k += T) add[k] = 0.0f;
    const float m = a.norm_in[2 * i], L = a.norm_in[2 * i + 1];
    float G = 0.0f, R = 0.0f;  // the gradients, and those that name columns of another score than m
    for (int p0 = 0; p0 < a.P; p0 += T) {
        const int p = p0 + (int)threadIdx.x;
        float xt;
        int c = target_of<E>(a, i, p, xt);
        float g = 0.0f;
        if (xt != -__builtin_inff()) g = a.g_logp[i * a.P + p];
        else c = -1;
        G += g;
        if (xt != m) R += g;
        const int at = c >= c0 && c - c0 < Y::kColumns ? c - c0 : -1;
        __syncthreads();  // add is zeroed, the last targets are added
        cols[threadIdx.x] = at;
        grads[threadIdx.x] = g;
        __syncthreads();
        if (threadIdx.x < 64) {
            const int lane = threadIdx.x;
            for (int q = 0; q < T && p0 + q < a.P; q += 64) {
                const int to = cols[q + lane];
                // a column that several of the 64 name is added to in their order: a lane
                // waits for as many rounds as lower lanes name its column
                int turn = to >= 0 ? 0 : -1;
                for (uint64_t left = __ballot(to >= 0); left != 0; left &= left - 1) {
                    const int l = __builtin_ctzll(left), c_l = __builtin_amdgcn_readlane(to, l);
                    turn += to == c_l && l < lane;
                }
                for (int round = 0; __ballot(turn >= round); ++round) {
                    if (turn == round) add[to] += grads[q + lane];
                    lds_fence();
                }
            }
        }
    }
    // A column with p = exp(-L) above 0.6, the only one whose score is m: the difference of
    // the gradients that name it, G - R, and p G loses the digits of 1 - p, (1 - p) G - R does
    // not. It takes the place of the other in a row's only store, or is stored over it (512
    // rows of 100,000 columns 78.3 -> 78.4 us, if all are such rows 81; chosen before each of
    // the stores 85).
    const bool peaked = L >= 0.0f && L < 0.5f;  // (-Inf: no candidates)
    G = wave_reduce(G, AddOp{});
    put(red[0], G);
    if (peaked) {
        R = wave_reduce(R, AddOp{});
        put(red[1], R);
    }
    __syncthreads();
    G = joined(red[0], G, AddOp{});

    const float gh = a.g_entropy ? a.g_entropy[i] : 0.0f, H = a.g_entropy ? a.entropy_in[i] : 0.0f;
    float sure = 0.0f;
    if (peaked) {
        R = joined(red[1], R, AddOp{});
        sure = a.scale * (__builtin_fmaf(one_minus_exp(L), G, -R) - exp_neg(-L) * gh * (H - L));
    }
    const int n = a.Nd - c0;
#pragma unroll
    for (int g = 0; g < N / Y::V; ++g) {
        const int at = Y::place(g * Y::V);
        float y[Y::V];
#pragma unroll
        for (int e = 0; e < Y::V; ++e) {
            const float v = x[g * Y::V + e];
            const float lp = floor_z(__builtin_fmaf(a.scale, v - m, -L));
            const float p = exp_neg(lp);
            const float d = a.scale * (add[at + e] - p * __builtin_fmaf(gh, lp + H, G));
            y[e] = v == -__builtin_inff() ? 0.0f : d;
        }
        if constexpr (N == Y::V) {
            if (peaked) {
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = x[e] == m ? sure : y[e];
            }
        }
        if (at < n) {
            if (a.out == kF32) store_columns<kF32, Y::V>(a.dX, i * a.Nd + c0 + at, n - at, y);
            else if (a.out == kBF16) store_columns<kBF16, Y::V>(a.dX, i * a.Nd + c0 + at, n - at, y);
            else store_columns<kF16, Y::V>(a.dX, i * a.Nd + c0 + at, n - at, y);
        }
    }
    if constexpr (N > Y::V) {
        if (peaked) {
            int mine = -1;
#pragma unroll
            for (int v = 0; v < N; ++v) mine = x[v] == m ? Y::place(v) : mine;
            const int64_t at = i * a.Nd + c0 + mine;
            if (mine >= 0) {
                if (a.out == kF32) ((float*)a.dX)[at] = sure;
                else ((uint16_t*)a.dX)[at] = (uint16_t)half_bits(a.out, sure);
            }
        }
    }
}

// One wave takes a row of as many columns as one load a lane brings, four waves one of
// four times as many: with 16 columns a lane the targets' ranks and the ordering of
// the best keep few waves busy (16 rows of 752 columns with 32 targets: one wave of 16
// columns a lane 32 us, four waves 10.7). Chunks of eight waves with 8 columns a lane
// are no faster than of four with 16 (32 x 100,000: 15.1 and 14.3 us).
template <int E>
void forward(const LogprobArgs& a, hipStream_t stream)
{
    constexpr int V = Layout<E, 64, kLpValues>::V;
    const dim3 rows((unsigned)a.Nq), chunks((unsigned)(a.Nq * a.chunks));
    if (a.Nd <= 64 * V) hipLaunchKernelGGL((logprob_part_kernel<E, 64, V, true>), rows, dim3(64), 0, stream, a);
    else if (a.Nd <= 256 * V) hipLaunchKernelGGL((logprob_part_kernel<E, 256, V, true>), rows, dim3(256), 0, stream, a);
    else if (a.chunks == 1) hipLaunchKernelGGL((logprob_part_kernel<E, 256, kLpValues, true>), rows, dim3(256), 0, stream, a);
    else {
        hipLaunchKernelGGL((logprob_part_kernel<E, 256, kLpValues, false>), chunks, dim3(256), 0, stream, a);
        hipLaunchKernelGGL((logprob_join_kernel<E>), rows, dim3(kJoinThreads), 0, stream, a);
    }
}

template <int E>
void backward(const LogprobArgs& a, hipStream_t stream)
{
    constexpr int V = Layout<E, 64, kLpValues>::V;
    const dim3 rows((unsigned)a.Nq), chunks((unsigned)(a.Nq * a.chunks));
    if (a.Nd <= 64 * V) hipLaunchKernelGGL((logprob_bwd_kernel<E, 64, V>), rows, dim3(64), 0, stream, a);
    else if (a.Nd <= 64 * kLpValues) hipLaunchKernelGGL((logprob_bwd_kernel<E, 64, kLpValues>), rows, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL((logprob_bwd_kernel<E, 256, kLpValues>), chunks, dim3(256), 0, stream, a);
}

// A grid's threads stay below 2^32: launches of at most `rows` rows.
template <typename F>
hipError_t by_rows(LogprobArgs a, int64_t es, F once)
{
    const int64_t rows = (int64_t)(1 << 22) / a.chunks > 0 ? (1 << 22) / a.chunks : 1;
    for (int64_t left = a.Nq; left > 0; left -= rows) {
        a.Nq = left < rows ? left : rows;
        once(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.X = (const char*)a.X + rows * a.Nd * es;
        if (a.mask) a.mask += rows * a.Nd;
        if (a.targets) a.targets += rows * a.P;
        if (a.logp) a.logp += rows * a.P;
        if (a.rank) a.rank += rows * a.P;
        if (a.norm) a.norm += 2 * rows;
        if (a.entropy) a.entropy += rows;
        if (a.top_idx) a.top_idx += rows * a.K;
        if (a.top_logp) a.top_logp += rows * a.K;
        if (a.norm_in) a.norm_in += 2 * rows;
        if (a.entropy_in) a.entropy_in += rows;
        if (a.g_logp) a.g_logp += rows * a.P;
        if (a.g_entropy) a.g_entropy += rows;
        if (a.dX) a.dX = (char*)a.dX + rows * a.Nd * (a.out == kF32 ? 4 : 2);
        if (a.ws_sums) {
            a.ws_sums += 2 * rows * a.chunks;
            a.ws_cand += rows * a.chunks * a.cap;
            a.ws_top += rows * a.chunks;
            a.ws_rank += rows * a.chunks * a.P;
        }
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_logprob_fwd(int elem, LogprobArgs a, hipStream_t stream)
{
    return by_rows(a, elem == kF32 ? 4 : 2, [&](const LogprobArgs& x) {
        if (elem == kF32) forward<kF32>(x, stream);
        else if (elem == kBF16) forward<kBF16>(x, stream);
        else forward<kF16>(x, stream);
    });
}

hipError_t launch_logprob_bwd(int elem, LogprobArgs a, hipStream_t stream)
{
    return by_rows(a, elem == kF32 ? 4 : 2, [&](const LogprobArgs& x) {
        if (elem == kF32) backward<kF32>(x, stream);
        else if (elem == kBF16) backward<kBF16>(x, stream);
        else backward<kF16>(x, stream);
    });
}

}  // namespace maxsim
