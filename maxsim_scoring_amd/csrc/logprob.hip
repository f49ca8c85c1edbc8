// Log probabilities of given columns under the softmax of their row of scores,
// with ranks, entropy and the row's best columns, and their gradient, for gfx950.
//
// Forward. A row is cut into chunks of 4096 columns, one workgroup each, 16 columns
// a thread in registers, read once: the largest score, the sums of exp(z) and of
// exp(z) z against it, how many columns come before each target (a ballot and a
// bit count per register), and the candidates for the best columns. Rows of one
// chunk (one wave up to 1024 columns) finish there; otherwise a second launch joins
// the chunks of a row. Few long rows spread over the card in this way.
//
// Best columns. Scores map to 32-bit keys in float order, and with the column behind
// them to numbers that are all different, whose order is that of the output. A
// histogram of 256 equal bins between the chunk's least and largest key finds the
// bin of the k-th; it is cut into 256 again only while more than k + k/2 + 32 lie
// at or above its lower edge. What is left is ordered by counting, for each, how
// many are larger.
//
// exp is the hardware's 2^x with the rounding of x log2(e) put back (off by about
// 2^-23 relative); sums are float64, so that a row whose largest probability is
// close to 1 keeps its entropy.
//
// Backward. One pass, element-wise but for the targets: their gradients are added
// into a chunk of columns in LDS by one wave, in the order of the targets.
#include "logprob.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

constexpr int kBins = 256;
constexpr int kMaxCap = 2048;     // logprob_cap(1024) and more, a power of two
constexpr uint32_t kNanKey = 0xffffffffu;

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));

template <int E> constexpr int elem_bytes() { return E == kF32 ? 4 : 2; }

// Keys in float order; 0 for what is no candidate (its key would be that of -Inf
// or below), the largest for NaN. -0 ranks with +0.
__device__ __forceinline__ uint32_t key_of(float v)
{
    uint32_t b = __builtin_bit_cast(uint32_t, v);
    if (v != v) return kNanKey;
    if (v == -__builtin_inff()) return 0;
    if (v == 0.0f) b = 0;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// The score of a key, -Inf of 0.
__device__ __forceinline__ float score_of(uint32_t k)
{
    if (k == 0) return -__builtin_inff();
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
__device__ __forceinline__ float floor_z(float z) { return z < -200.0f ? -200.0f : z; }

// A row's columns c0 + place, 16 per thread of T: value v of a thread is column
// place(v) of the chunk; V consecutive ones come in one load.
template <int E, int T>
struct Layout {
    static constexpr int V = E == kF32 ? 4 : 8;
    static constexpr int kColumns = T * kLpValues;
    __device__ static __forceinline__ int place(int v) { return ((v / V) * T + (int)threadIdx.x) * V + v % V; }
};

// The thread's columns of row i from c0 on: NaN-free loading of what exists and is
// not masked, -Inf elsewhere.
template <int E, int T>
__device__ __forceinline__ void load_columns(const LogprobArgs& a, int64_t i, int c0, float (&x)[kLpValues])
{
    typedef Layout<E, T> Y;
    const int n = a.Nd - c0 < Y::kColumns ? a.Nd - c0 : Y::kColumns;
    const char* p = (const char*)a.X + (i * a.Nd + c0) * elem_bytes<E>();
    const uint8_t* mp = a.mask ? a.mask + i * a.Nd + c0 : nullptr;
#pragma unroll
    for (int g = 0; g < kLpValues / Y::V; ++g) {
        const int at = Y::place(g * Y::V);
        u32x4 w = {0, 0, 0, 0};
        uint32_t keep[Y::V / 4];
#pragma unroll
        for (int k = 0; k < Y::V / 4; ++k) keep[k] = 0;
        if (at + Y::V <= n) {
            w = *(const u32x4_any*)(p + (int64_t)at * elem_bytes<E>());
#pragma unroll
            for (int k = 0; k < Y::V / 4; ++k) keep[k] = mp ? *(const u32_any*)(mp + at + 4 * k) : 0x01010101u;
        } else {
#pragma unroll
            for (int e = 0; e < Y::V; ++e) {
                if (at + e >= n) continue;
                if constexpr (E == kF32) w[e] = ((const uint32_t*)p)[at + e];
                else w[e / 2] |= (uint32_t)((const uint16_t*)p)[at + e] << (16 * (e & 1));
                keep[e / 4] |= (mp ? (uint32_t)mp[at + e] : 1u) << (8 * (e & 3));
            }
        }
#pragma unroll
        for (int e = 0; e < Y::V; ++e) {
            float v;
            if constexpr (E == kF32) v = as_float(w[e]);
            else {
                const uint32_t bits = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
                v = E == kBF16 ? __builtin_bit_cast(float, bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
            }
            x[g * Y::V + e] = (keep[e / 4] >> (8 * (e & 3))) & 0xffu ? v : -__builtin_inff();
        }
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

// Reductions over a workgroup of T threads, the same result in every thread. `red`
// is LDS of T / 64 values; a barrier lies before its next use.
template <int T, typename V, typename OP>
__device__ __forceinline__ V block_reduce(V v, V* red, OP op)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v = op(v, __shfl_xor(v, m, 64));
    if constexpr (T > 64) {
        __syncthreads();
        if (lane_id() == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) v = op(v, red[w]);
    }
    return v;
}
struct AddOp { template <typename V> __device__ __forceinline__ V operator()(V a, V b) const { return a + b; } };
struct MaxOp { template <typename V> __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; } };

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

// A bound such that at least K and at most cap of a set of numbers, all different
// and between lo and hi, are at or above it (the set has more than cap, cap >= K).
// each(f) calls f(number) for each of this thread's. hist: LDS of kBins + 2.
template <int T, typename Each>
__device__ __forceinline__ uint64_t select_bound(Each each, uint32_t K, uint32_t cap, uint64_t lo, uint64_t hi, uint32_t* hist)
{
    int width = 64 - __builtin_clzll((hi - lo) | 1);  // [lo, lo + 2^width) holds them
    uint32_t above = 0;                               // numbers beyond that range
    for (;;) {
        const int shift = width > 8 ? width - 8 : 0;
        const uint64_t end = width < 64 ? lo + ((uint64_t)1 << width) : 0;  // 0: none
        __syncthreads();
        for (int k = threadIdx.x; k < kBins; k += T) hist[k] = 0;
        __syncthreads();
        each([&](uint64_t o) {
            if (o >= lo && (end == 0 || o < end)) atomicAdd(&hist[(o - lo) >> shift], 1u);
        });
        __syncthreads();
        if (threadIdx.x < 64) {
            // lane 0 holds the top bins; the bin where the count from the top reaches K
            const int lane = threadIdx.x;
            uint32_t c[4], mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) mine += c[e] = hist[255 - (4 * lane + e)];
            uint32_t incl = mine;
#pragma unroll
            for (int off = 1; off < 64; off *= 2) {
                const uint32_t v = __shfl_up(incl, off, 64);
                if (lane >= off) incl += v;
            }
            uint32_t before = above + incl - mine;
            uint32_t bin = 0, over = 0, upto = 0;
            bool found = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (before < K && K <= before + c[e]) {
                    bin = (uint32_t)(255 - (4 * lane + e));
                    over = before;
                    upto = before + c[e];
                    found = true;
                }
                before += c[e];
            }
            if (found) {  // one lane; all lanes have read their bins
                hist[kBins] = bin;
                hist[kBins + 1] = over;
                hist[kBins + 2] = upto;
            }
        }
        __syncthreads();
        lo += (uint64_t)hist[kBins] << shift;
        above = hist[kBins + 1];
        if (hist[kBins + 2] <= cap || shift == 0) return lo;
        width = shift;
    }
}

// Writes the K best of n <= kMaxCap numbers of cand (LDS) in order; z and L give
// their log probabilities.
template <int T>
__device__ __forceinline__ void write_best(const LogprobArgs& a, int64_t i, const uint64_t* cand, int n, float m, double L)
{
    for (int e = threadIdx.x; e < n; e += T) {
        const uint64_t mine = cand[e];
        int place = 0;
        for (int k = 0; k < n; ++k) place += cand[k] > mine;
        if (place < a.K) {
            const float x = score_of((uint32_t)(mine >> a.cbits));
            a.top_idx[i * a.K + place] = column_of(mine, a.cbits);
            a.top_logp[i * a.K + place] = (float)((double)(a.scale * (x - m)) - L);
        }
    }
    for (int e = n + threadIdx.x; e < a.K; e += T) {
        a.top_idx[i * a.K + e] = -1;
        a.top_logp[i * a.K + e] = L == L ? -__builtin_inff() : (float)L;
    }
}

// A row's statistics. A NaN or +Inf among the candidates makes the sums NaN, and
// with them every float output of the row.
__device__ __forceinline__ void write_stats(const LogprobArgs& a, int64_t i, float m, double sum, double sum_z, double L)
{
    a.norm[2 * i] = L == L ? m : __builtin_nanf("");
    a.norm[2 * i + 1] = (float)L;
    if (a.entropy) a.entropy[i] = sum == 0.0 ? 0.0f : (float)(L - sum_z / sum);
}

// Target p of a row, `before` candidates before it.
template <int E>
__device__ __forceinline__ void write_target(const LogprobArgs& a, int64_t i, int p, uint32_t before, float m, double L)
{
    const int c = a.targets[i * a.P + p];
    const bool named = c >= 0 && c < a.Nd;
    const float x = named ? load_one<E>(a, i, c) : -__builtin_inff();
    const bool in = x != -__builtin_inff();
    float lp = named ? x : 0.0f;
    if (in || L != L) lp = (float)((double)(a.scale * (x - m)) - L);
    a.logp[i * a.P + p] = lp;
    if (a.rank) a.rank[i * a.P + p] = in ? (int)before : -1;
}

// One chunk of a row. WHOLE: the row's only one.
template <int E, int T, bool WHOLE>
__global__ __launch_bounds__(T) void logprob_part_kernel(LogprobArgs a)
{
    typedef Layout<E, T> Y;
    __shared__ uint32_t hist[kBins + 4];
    __shared__ uint64_t cand[WHOLE ? kMaxCap : 1];
    __shared__ uint32_t red_key[4], counter;
    __shared__ double red_sum[4];
    __shared__ uint32_t counts[4][64];

    const int64_t unit = blockIdx.x, i = WHOLE ? unit : unit / a.chunks;
    const int c0 = WHOLE ? 0 : (int)(unit % a.chunks) * Y::kColumns;
    float x[kLpValues];
    load_columns<E, T>(a, i, c0, x);

    uint32_t key[kLpValues], top = 0, least = kNanKey;
    int have = 0;
#pragma unroll
    for (int v = 0; v < kLpValues; ++v) {
        key[v] = key_of(x[v]);
        top = key[v] > top ? key[v] : top;
        if (key[v] != 0) {
            least = key[v] < least ? key[v] : least;
            ++have;
        }
    }
    top = block_reduce<T>(top, red_key, MaxOp{});
    const float m = score_of(top);
    double sum = 0.0, sum_z = 0.0;
#pragma unroll
    for (int v = 0; v < kLpValues; ++v) {
        const float z = floor_z(a.scale * (x[v] - m));
        const float e = exp_neg(z);
        if (key[v] != 0) {
            sum += (double)e;
            sum_z = __builtin_fma((double)e, (double)z, sum_z);
        }
    }
    sum = block_reduce<T>(sum, red_sum, AddOp{});
    sum_z = block_reduce<T>(sum_z, red_sum, AddOp{});

    // ---- how many come before each target, 64 targets at a time --------------
    const int wave = threadIdx.x >> 6, lane = lane_id();
    auto count_before = [&](int p0, uint32_t& got) {  // got: that of target p0 + lane, in wave 0
        const int np = a.P - p0 < 64 ? a.P - p0 : 64;
        // every lane looks its target up; then one target after another
        const int c = lane < np ? a.targets[i * a.P + p0 + lane] : -1;
        uint32_t kt = 0;
        if (c >= 0 && c < a.Nd) kt = key_of(load_one<E>(a, i, c));
        uint32_t n_mine = 0;
        for (int p = 0; p < np; ++p) {
            const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)kt, p);
            const int t = __builtin_amdgcn_readlane(c, p) - c0;  // relative to the chunk
            if (k == 0) continue;
            // equal scores come before the target if their column does: none of a
            // chunk behind it, all of one in front of it
            uint32_t n = 0;
            auto count = [&](auto before) {
#pragma unroll
                for (int v = 0; v < kLpValues; ++v) n += (uint32_t)__builtin_popcountll(__ballot(before(v)));
            };
            if (t < 0) count([&](int v) { return key[v] > k; });
            else if (t >= Y::kColumns) count([&](int v) { return key[v] >= k; });
            else count([&](int v) { return key[v] > k || (key[v] == k && Y::place(v) < t); });
            n_mine = lane == p ? n : n_mine;
        }
        got = n_mine;
        if constexpr (T > 64) {
            __syncthreads();  // the last targets' counts are read
            counts[wave][lane] = n_mine;
            __syncthreads();
            got = counts[0][lane] + counts[1][lane] + counts[2][lane] + counts[3][lane];
        }
    };

    const double L = WHOLE ? log(sum) : 0.0;
    if constexpr (WHOLE) {
        if (threadIdx.x == 0) write_stats(a, i, m, sum, sum_z, L);
        for (int p0 = 0; p0 < a.P; p0 += 64) {
            uint32_t got = 0;
            if (a.rank) count_before(p0, got);
            if (wave == 0 && p0 + lane < a.P) write_target<E>(a, i, p0 + lane, got, m, L);
        }
    } else {
        if (threadIdx.x == 0) {
            a.ws_top[unit] = top;
            a.ws_sums[2 * unit] = sum;
            a.ws_sums[2 * unit + 1] = sum_z;
        }
        if (a.rank) {
            for (int p0 = 0; p0 < a.P; p0 += 64) {
                uint32_t got;
                count_before(p0, got);
                if (wave == 0 && p0 + lane < a.P) a.ws_rank[unit * a.P + p0 + lane] = got;
            }
        }
    }
    if (a.K == 0) return;

    // ---- candidates for the best columns --------------------------------------
    have = (int)block_reduce<T>((uint32_t)have, red_key, AddOp{});
    least = ~block_reduce<T>(~least, red_key, MaxOp{});
    auto number = [&](int v) { return order_of(key[v], c0 + Y::place(v), a.cbits); };
    uint64_t bound = 0;
    if (have > a.cap)
        bound = select_bound<T>(
            [&](auto f) {
#pragma unroll
                for (int v = 0; v < kLpValues; ++v)
                    if (key[v] != 0) f(number(v));
            },
            (uint32_t)a.K, (uint32_t)a.cap, (uint64_t)least << a.cbits, order_of(top, 0, a.cbits), hist);
    if (threadIdx.x == 0) counter = 0;
    __syncthreads();
    uint64_t* to = WHOLE ? cand : a.ws_cand + unit * a.cap;
    // their places depend on the waves' timing, the outputs do not: they are ordered later
#pragma unroll
    for (int v = 0; v < kLpValues; ++v) {
        const bool take = key[v] != 0 && number(v) >= bound;
        if (take) {
            const uint32_t at = atomicAdd(&counter, 1u);
            if (at < (uint32_t)a.cap) to[at] = number(v);
        }
    }
    __syncthreads();
    if constexpr (WHOLE) write_best<T>(a, i, cand, (int)counter, m, L);
    else if (threadIdx.x == 0) a.ws_count[unit] = counter;
}

// Joins the chunks of a row.
template <int E>
__global__ __launch_bounds__(256) void logprob_join_kernel(LogprobArgs a)
{
    constexpr int T = 256;
    __shared__ uint32_t hist[kBins + 4];
    __shared__ uint64_t cand[kMaxCap];
    __shared__ uint32_t red_key[4], counter;
    __shared__ double red_sum[4];

    const int64_t i = blockIdx.x, u0 = i * a.chunks;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < a.chunks; c += T) top = MaxOp{}(top, a.ws_top[u0 + c]);
    top = block_reduce<T>(top, red_key, MaxOp{});
    const float m = score_of(top);
    double sum = 0.0, sum_z = 0.0;
    for (int c = threadIdx.x; c < a.chunks; c += T) {
        const double s = a.ws_sums[2 * (u0 + c)], sz = a.ws_sums[2 * (u0 + c) + 1];
        const uint32_t k = a.ws_top[u0 + c];
        if (k == 0) continue;
        const float z = floor_z(a.scale * (score_of(k) - m));  // the chunk's largest against the row's
        const double e = (double)exp_neg(z);
        sum = __builtin_fma(e, s, sum);
        sum_z = __builtin_fma(e, __builtin_fma((double)z, s, sz), sum_z);
    }
    sum = block_reduce<T>(sum, red_sum, AddOp{});
    sum_z = block_reduce<T>(sum_z, red_sum, AddOp{});
    const double L = log(sum);
    if (threadIdx.x == 0) write_stats(a, i, m, sum, sum_z, L);
    for (int p = threadIdx.x; p < a.P; p += T) {
        uint32_t n = 0;
        if (a.rank)
            for (int c = 0; c < a.chunks; ++c) n += a.ws_rank[(u0 + c) * a.P + p];
        write_target<E>(a, i, p, n, m, L);
    }
    if (a.K == 0) return;

    uint32_t total = 0;
    for (int c = threadIdx.x; c < a.chunks; c += T) total += a.ws_count[u0 + c];
    total = block_reduce<T>(total, red_key, AddOp{});
    auto each = [&](auto f) {
        for (int c = threadIdx.x >> 6; c < a.chunks; c += T / 64) {
            const int n = (int)a.ws_count[u0 + c];
            for (int e = lane_id(); e < n; e += 64) f(a.ws_cand[(u0 + c) * a.cap + e]);
        }
    };
    uint64_t bound = 0;
    if (total > (uint32_t)a.cap) {
        uint64_t least = ~(uint64_t)0;
        each([&](uint64_t o) { least = o < least ? o : least; });
        __shared__ uint64_t red_o[4];
        least = ~block_reduce<T>(~least, red_o, MaxOp{});
        bound = select_bound<T>(each, (uint32_t)a.K, (uint32_t)a.cap, least, order_of(top, 0, a.cbits), hist);
    }
    if (threadIdx.x == 0) counter = 0;
    __syncthreads();
    each([&](uint64_t o) {
        if (o >= bound) {
            const uint32_t at = atomicAdd(&counter, 1u);
            if (at < (uint32_t)a.cap) cand[at] = o;
        }
    });
    __syncthreads();
    write_best<T>(a, i, cand, (int)counter, m, L);
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

template <int E, int T>
__global__ __launch_bounds__(T) void logprob_bwd_kernel(LogprobArgs a)
{
    typedef Layout<E, T> Y;
    __shared__ float add[Y::kColumns];  // the targets' gradients, by column
    __shared__ int cols[T];
    __shared__ float grads[T];
    __shared__ float red[4];

    const int64_t unit = blockIdx.x, i = unit / a.chunks;
    const int c0 = (int)(unit % a.chunks) * Y::kColumns;
    float x[kLpValues];
    load_columns<E, T>(a, i, c0, x);
    for (int k = threadIdx.x; k < Y::kColumns; k += T) add[k] = 0.0f;
    float G = 0.0f;
    for (int p0 = 0; p0 < a.P; p0 += T) {
        const int p = p0 + (int)threadIdx.x;
        int c = p < a.P ? a.targets[i * a.P + p] : -1;
        float g = 0.0f;
        if (c >= 0 && c < a.Nd && load_one<E>(a, i, c) != -__builtin_inff()) g = a.g_logp[i * a.P + p];
        else c = -1;
        G += g;
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
    G = block_reduce<T>(G, red, AddOp{});
    __syncthreads();

    const float m = a.norm_in[2 * i], L = a.norm_in[2 * i + 1];
    const float gh = a.g_entropy ? a.g_entropy[i] : 0.0f, H = a.g_entropy ? a.entropy_in[i] : 0.0f;
    const int n = a.Nd - c0;
#pragma unroll
    for (int g = 0; g < kLpValues / Y::V; ++g) {
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
        if (at < n) {
            if (a.out == kF32) store_columns<kF32, Y::V>(a.dX, i * a.Nd + c0 + at, n - at, y);
            else if (a.out == kBF16) store_columns<kBF16, Y::V>(a.dX, i * a.Nd + c0 + at, n - at, y);
            else store_columns<kF16, Y::V>(a.dX, i * a.Nd + c0 + at, n - at, y);
        }
    }
}

template <int E>
void forward(const LogprobArgs& a, hipStream_t stream)
{
    if (a.Nd <= 64 * kLpValues) {
        hipLaunchKernelGGL((logprob_part_kernel<E, 64, true>), dim3((unsigned)a.Nq), dim3(64), 0, stream, a);
    } else if (a.chunks == 1) {
        hipLaunchKernelGGL((logprob_part_kernel<E, 256, true>), dim3((unsigned)a.Nq), dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL((logprob_part_kernel<E, 256, false>), dim3((unsigned)(a.Nq * a.chunks)), dim3(256), 0, stream, a);
        hipLaunchKernelGGL((logprob_join_kernel<E>), dim3((unsigned)a.Nq), dim3(256), 0, stream, a);
    }
}

template <int E>
void backward(const LogprobArgs& a, hipStream_t stream)
{
    if (a.Nd <= 64 * kLpValues) hipLaunchKernelGGL((logprob_bwd_kernel<E, 64>), dim3((unsigned)a.Nq), dim3(64), 0, stream, a);
    else hipLaunchKernelGGL((logprob_bwd_kernel<E, 256>), dim3((unsigned)(a.Nq * a.chunks)), dim3(256), 0, stream, a);
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
            a.ws_count += rows * a.chunks;
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
