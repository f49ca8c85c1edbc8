// Product of microscaled 4-bit rows with microscaled 4-bit weights, for gfx950.
//
//   Y[t,n] = sum over blocks b of 2^(ea[t,b] + ew[n,b]) <A[t,b], W[n,b]> + bias[n]
//
// The block-scaled MFMA multiplies both powers of two itself, so the codes go
// from memory to the matrix cores as they are, with one exponent byte for every 16
// bytes of codes. As in the 8-bit product the result is formed transposed, W . A^T,
// with the channels in an order that leaves 16 consecutive ones in a lane.
//
// tile_mx4_kernel: BT tokens x BN channels per workgroup; steps of 128 bytes of
// both operands (8 blocks) stream through a ring in LDS by direct-to-LDS loads,
// 16-byte chunks swizzled against bank conflicts, the 8 exponents of each row
// beside them. Lane half h takes blocks 4 h .. 4 h + 3 of a step (any order of k
// serves as long as both operands share it), so that its four exponents are one
// aligned word and the MFMA's byte selector picks them.
// few_mx4_kernel: a few tokens. W is the traffic; fragments go straight from
// memory to registers, 8 waves split k, and LDS joins their sums.
//
// 8192 x 4096 x 4096 to bf16 takes 80 us (3.4 PFLOP/s; the profiler's median is 81 to
// 84), 8192 x 8192 x 8192 270 us (4.1), where a loop of these MFMAs alone reaches 4.6
// to 5.1 on such values (power is the limit; 7.5 on zeros): about 20 us go to filling
// the pipeline and to 67 MB of outputs, the rest grows with k at 4.4 PFLOP/s. One token
// by 4096 x 4096: 5.0 us for 8.9 MB, most of it the latency of a launch and of one chain
// of loads. Not faster were tiles of 128 x 128 a wave (94 against 87 us at the time),
// workgroups that take several 256 x 256 tiles, and outputs turned through LDS.
#include "mx4_common.hpp"
#include "kernels.hpp"

namespace maxsim {

namespace {

typedef uint64_t u64_any __attribute__((aligned(1)));

// Writes a wave's NT x 32 channels of TT x 32 tokens, from channel n0 + wn * NT * 32
// and token t0 + a_row on. ring: LDS of at least 32 x (NT * 32 + 4) floats per
// wave, free to overwrite.
template <int NT, int TT>
__device__ __forceinline__ void store_tile(const Mx4LinearArgs& a, const f32x16 (&acc)[NT][TT], const float* bs,
                                           int64_t t0, int n0, int a_row, int wn, int wave, uint8_t* ring)
{
    const int lane = lane_id(), half = lane >> 5;
    if (a.N & 3) {
        // rows at any address: the wave turns its tokens x channels through LDS, so
        // that lanes store neighbouring channels
        constexpr int kCols = NT * 32, kStride = kCols + 4;
        float* mine = (float*)ring + wave * 32 * kStride;
        const int n_base = wn * kCols;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int64_t tile = t0 + a_row + j * 32;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int n = i * 32 + half * 16 + e;
                    mine[(lane & 31) * kStride + n] = acc[i][j][e] + bs[n_base + n];
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
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = t0 + a_row + j * 32 + (lane & 31);
        if (t >= a.T) continue;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = (wn * NT + i) * 32 + half * 16;
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = acc[i][j][e] + bs[n + e];
            store_run<16>(a.Y, a.out, t, n0 + n, a.N, y);
        }
    }
}

// Position to tile: consecutive workgroups go to the 8 XCDs in turn, so each XCD
// takes a contiguous run of tiles, walked in bands of 8 token tiles, whose
// operands the XCD's L2 then holds.
__device__ __forceinline__ void tile_of(const Mx4LinearArgs& a, int b, int BT, int BN, int64_t& t0, int& n0)
{
    const int nwg = a.tiles_t * a.tiles_n;
    const int q = nwg >> 3, r = nwg & 7, x = b & 7;
    const int id = x * q + (x < r ? x : r) + (b >> 3);
    const int per = 8 * a.tiles_n, band = id / per, in = id - band * per;
    const int left = a.tiles_t - band * 8, high = left < 8 ? left : 8;
    t0 = (int64_t)(band * 8 + in % high) * BT;
    n0 = in / high * BN;
}

template <int BT, int BN, int WT, int WN, int ST>
struct Tile {
    static constexpr int KB = 128;                    // bytes of codes of a row and step
    static constexpr int kWaves = WT * WN;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int TT = BT / WT / 32;           // 32-token column tiles per wave
    static constexpr int NT = BN / WN / 32;           // 32-channel row tiles per wave
    static constexpr int kRows = BT + BN;
    static constexpr int kCodes = kRows * KB;
    static constexpr int kStage = kCodes + kRows * 8;  // the exponents behind the codes
    static constexpr int kPerWave = kRows / 8 / kWaves;     // wave-wide loads of codes: 8 rows each
    static constexpr int kScales = (kRows / 32 + kWaves - 1) / kWaves;  // and of exponents: 32 rows each
    static_assert(BT % 32 == 0 && BN % 32 == 0 && kRows % (8 * kWaves) == 0, "a load stays inside one operand, every wave has as many");
    static_assert(kWaves * 32 * (NT * 32 + 4) * 4 <= ST * kStage, "the ring holds a turned output");
};

// One step's MFMAs: the wave's channels x tokens.
template <typename C>
__device__ __forceinline__ void multiply(const uint8_t* buf, int w_row, int a_row, f32x16 (&acc)[C::NT][C::TT])
{
    const int l = lane_id() & 31, h = lane_id() >> 5;
    const uint8_t* sc = buf + C::kCodes;
    int sw[C::NT], sx[C::TT];
#pragma unroll
    for (int i = 0; i < C::NT; ++i) sw[i] = *(const int*)(sc + (w_row + i * 32 + l) * 8 + h * 4);
#pragma unroll
    for (int i = 0; i < C::TT; ++i) sx[i] = *(const int*)(sc + (a_row + i * 32 + l) * 8 + h * 4);
    static_for<0, 4>([&](auto ks) {
        const int off = place<C::KB>(l, 4 * h + ks) * 16 + l * C::KB;
        i32x4 w[C::NT], x[C::TT];
#pragma unroll
        for (int i = 0; i < C::NT; ++i) w[i] = *(const i32x4*)(buf + (w_row + i * 32) * C::KB + off);
#pragma unroll
        for (int i = 0; i < C::TT; ++i) x[i] = *(const i32x4*)(buf + (a_row + i * 32) * C::KB + off);
#pragma unroll
        for (int i = 0; i < C::NT; ++i)
#pragma unroll
            for (int j = 0; j < C::TT; ++j) acc[i][j] = mfma32_mx4<ks, ks>(w[i], sw[i], x[j], sx[j], acc[i][j]);
    });
}

// WORDS: the exponents of a row come in aligned words (nb is a multiple of 4) and
// go to LDS directly; otherwise they pass through registers (8192 x 4096 x 4096 80 us,
// 8192 x 4096 x 4000 98).
// MANY: a workgroup takes every gridDim.x-th tile, and loads the first steps of the
// next one before it stores the outputs of this one.
template <int BT, int BN, int WT, int WN, int ST, bool WORDS, bool MANY>
__global__ __launch_bounds__(WT* WN * 64) void tile_mx4_kernel(Mx4LinearArgs a)
{
    typedef Tile<BT, BN, WT, WN, ST> C;
    __shared__ __align__(1024) uint8_t ring[ST * C::kStage];
    __shared__ __align__(16) float bias[2][BN];

    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int wt = wave / WN, wn = wave % WN;
    const int a_row = wt * C::TT * 32, w_row = BT + wn * C::NT * 32;
    const int row_bytes = a.nb * 16, nk = a.nb / 8;  // whole steps
    const int tiles = a.tiles_t * a.tiles_n;
    constexpr int L = C::kPerWave + (WORDS ? C::kScales : 0);  // a wave's loads of a step
    constexpr int S = C::NT * C::TT * 2;                       // stores of a whole tile, at least

    // ---- the tile whose operands are being loaded --------------------------------
    int64_t t0;
    int n0, rows_t, rows_n;
    const uint8_t *A, *W, *SA, *SW;
    // The wave's loads: load j brings 8 rows of codes, one chunk per lane, or (the
    // exponents) 32 rows, one word per lane.
    uint32_t voff[C::kPerWave], soff[C::kScales];
    auto row_of = [&](int j) { return (wave * C::kPerWave + j) * 8; };
    auto srow_of = [&](int j) {  // a spare load repeats the last
        const int at = (wave * C::kScales + j) * 32;
        return at < C::kRows ? at : C::kRows - 32;
    };
    // Which row of its operand a row of the stage holds. Rows past the end of an
    // operand repeat its last row; what they give is not stored.
    auto local = [](int r, int rows_t, int rows_n) {
        const bool isA = r < BT;
        const int row = isA ? r : channel_of(r - BT), last = (isA ? rows_t : rows_n) - 1;
        return row < last ? row : last;
    };
    auto enter = [&](int at, float* bs) {
        tile_of(a, at, BT, BN, t0, n0);
        rows_t = (int)(a.T - t0 < BT ? a.T - t0 : BT);
        rows_n = a.N - n0 < BN ? a.N - n0 : BN;
        A = a.A + t0 * row_bytes;
        W = a.W + (int64_t)n0 * row_bytes;
        SA = a.a_scale + t0 * a.nb;
        SW = a.w_scale + (int64_t)n0 * a.nb;
        for (int i = threadIdx.x; i < BN; i += C::kThreads) bs[i] = a.bias && i < rows_n ? a.bias[n0 + i] : 0.0f;
#pragma unroll
        for (int j = 0; j < C::kPerWave; ++j) {
            const int r = row_of(j) + lane / 8;
            voff[j] = (uint32_t)local(r, rows_t, rows_n) * (uint32_t)row_bytes + (uint32_t)place<C::KB>(r, lane % 8) * 16;
        }
#pragma unroll
        for (int j = 0; j < C::kScales; ++j)
            soff[j] = (uint32_t)local(srow_of(j) + lane / 2, rows_t, rows_n) * (uint32_t)a.nb + (uint32_t)(lane & 1) * 4;
    };
    const uint32_t ring0 = lds_addr(ring);
    auto issue = [&](int i) {
        const uint32_t at = ring0 + (uint32_t)(i % ST) * C::kStage;
        const uint8_t* pa = A + (int64_t)i * C::KB;
        const uint8_t* pw = W + (int64_t)i * C::KB;
#pragma unroll
        for (int j = 0; j < C::kPerWave; ++j) {
            const int base = row_of(j);
            dma_lds16(uniform_ptr(base < BT ? pa : pw), voff[j], (uint32_t)uniform((int)(at + base * C::KB)));
        }
        if constexpr (WORDS) {
#pragma unroll
            for (int j = 0; j < C::kScales; ++j) {
                const int base = srow_of(j);
                dma_lds4(uniform_ptr((base < BT ? SA : SW) + i * 8), soff[j], (uint32_t)uniform((int)(at + C::kCodes + base * 8)));
            }
        }
    };
    auto fill = [&] {
#pragma unroll
        for (int s = 0; s < ST; ++s)
            if (s < nk) issue(s);
    };
    // Exponents of step i through registers: in the last step the blocks behind the
    // last one count as 2^0 (their codes are zeros).
    auto scales = [=, nb = a.nb](const uint8_t* sa, const uint8_t* sw, int rt, int rn, int i, uint8_t* buf) {
        for (int r = threadIdx.x; r < C::kRows; r += C::kThreads) {
            const uint8_t* p = (r < BT ? sa : sw) + (int64_t)local(r, rt, rn) * nb + 8 * i;
            uint64_t w = 0;
            if (8 * i + 8 <= nb) {
                w = *(const u64_any*)p;
            } else {
#pragma unroll
                for (int b = 0; b < 8; ++b) w |= (uint64_t)(8 * i + b < nb ? p[b] : 127) << (8 * b);
            }
            *(uint64_t*)(buf + C::kCodes + r * 8) = w;
        }
    };

    int at = blockIdx.x, turn = 0;
    bool stored = false;  // S stores or more of the tile before are behind the first steps' loads
    enter(at, bias[0]);
    fill();
    for (;;) {
        f32x16 acc[C::NT][C::TT];
#pragma unroll
        for (int i = 0; i < C::NT; ++i)
#pragma unroll
            for (int j = 0; j < C::TT; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        for (int i = 0; i < nk; ++i) {
            uint8_t* buf = ring + (i % ST) * C::kStage;
            if constexpr (!WORDS) scales(SA, SW, rows_t, rows_n, i, buf);  // all waves have read what it held
            // Step i has landed if at most the loads behind its own are out: those of the ST - 1
            // (at first) or ST - 2 later steps, and the stores. (The counter goes down in the
            // order of issue, loads and stores alike.)
            if (MANY && ST == 2 && WORDS && stored && i < 2) {
                if (i == 0 && nk > 1) wait_vmcnt<L + S>();
                else wait_vmcnt<S>();
            } else if (WORDS && i == 0 && nk >= ST) wait_vmcnt<(ST - 1) * L>();
            else if (WORDS && ST > 2 && i > 0 && i + ST - 2 < nk) wait_vmcnt<(ST - 2) * L>();
            else wait_vmcnt<0>();
            block_barrier();  // all waves' loads of step i landed; step i - 1 is read
            if (i > 0 && i + ST - 1 < nk) issue(i + ST - 1);
            multiply<C>(buf, w_row, a_row, acc);
        }
        if (a.nb & 7) {
            // the blocks behind the last whole step, zeros behind them; step nk - ST, which
            // held this buffer, was read before the last barrier
            uint8_t* buf = ring + (nk % ST) * C::kStage;
            for (int c = threadIdx.x; c < C::kRows * 8; c += C::kThreads) {
                const int r = c / 8, b = nk * 8 + c % 8;
                const uint8_t* src = (r < BT ? A : W) + (int64_t)local(r, rows_t, rows_n) * row_bytes;
                *(i32x4*)(buf + r * C::KB + place<C::KB>(r, c % 8) * 16) = b < a.nb ? *(const i32x4*)(src + b * 16) : i32x4{};
            }
            scales(SA, SW, rows_t, rows_n, nk, buf);
            block_barrier();
            multiply<C>(buf, w_row, a_row, acc);
        }
        __syncthreads();  // the ring is read, the bias written
        const int64_t t_done = t0;
        const int n_done = n0;
        const float* bs = bias[turn];
        const bool more = MANY && at + (int)gridDim.x < tiles;
        const bool turned = (a.N & 3) != 0;  // outputs go through the ring
        if (more) {
            stored = !turned && rows_t == BT && rows_n == BN;
            at += gridDim.x;
            turn ^= 1;
            enter(at, bias[turn]);
            if (!turned) fill();
        }
        store_tile<C::NT, C::TT>(a, acc, bs, t_done, n_done, a_row, wn, wave, ring);
        if (!more) break;
        if (turned) {
            __syncthreads();
            fill();
        }
    }
}

// TT x 16 tokens by 16 channels per workgroup; KW waves split k in steps of 4 blocks.
template <int TT, int KW, bool WORDS>
__global__ __launch_bounds__(KW * 64) void few_mx4_kernel(Mx4LinearArgs a)
{
    __shared__ f32x4 sums[KW > 1 ? (KW - 1) * TT * 64 : 1];
    const int kw = uniform((int)threadIdx.x >> 6), lane = lane_id(), row = lane & 15, quarter = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int64_t t0 = (int64_t)blockIdx.y * (TT * 16);
    const int row_bytes = a.nb * 16;

    const int n = n0 + row < a.N ? n0 + row : a.N - 1;
    const uint8_t* wp = a.W + (int64_t)n * row_bytes;
    const uint8_t* ws = a.w_scale + (int64_t)n * a.nb;
    const uint8_t* xp[TT];
    const uint8_t* xs[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = t0 + j * 16 + row, at = t < a.T ? t : a.T - 1;
        xp[j] = a.A + at * row_bytes;
        xs[j] = a.a_scale + at * a.nb;
    }
    f32x4 acc[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = (a.nb + 3) / 4, per = (steps + KW - 1) / KW;
    const int s1 = (kw + 1) * per < steps ? (kw + 1) * per : steps;
    constexpr int U = 8;  // steps whose loads fly together
    for (int s = kw * per; s < s1; s += U) {
        i32x4 w[U], x[U][TT];
        int sw[U], sx[U][TT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = 4 * (s + u) + quarter;
            const bool in = s + u < s1 && b < a.nb;
            auto scale = [&](const uint8_t* p) -> int {
                if constexpr (WORDS) return in ? *(const int*)(p + (b & ~3)) : 0;
                else return in ? p[b] : 127;
            };
            w[u] = in ? *(const i32x4*)(wp + b * 16) : i32x4{};
            sw[u] = scale(ws);
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                x[u][j] = in ? *(const i32x4*)(xp[j] + b * 16) : i32x4{};
                sx[u][j] = scale(xs[j]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (WORDS) sw[u] = (int)((uint32_t)sw[u] >> (8 * quarter));
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                if constexpr (WORDS) sx[u][j] = (int)((uint32_t)sx[u][j] >> (8 * quarter));
                acc[j] = mfma16_mx4<0, 0>(w[u], sw[u], x[u][j], sx[u][j], acc[j]);
            }
        }
    }
    if constexpr (KW > 1) {
        if (kw > 0) {
#pragma unroll
            for (int j = 0; j < TT; ++j) sums[((kw - 1) * TT + j) * 64 + lane] = acc[j];
        }
        __syncthreads();
        if (kw > 0) return;
        for (int o = 0; o < KW - 1; ++o) {
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[j] += sums[(o * TT + j) * 64 + lane];
        }
    }
    const int c = n0 + quarter * 4;  // rows of the result: channels c .. c + 3
    float bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = a.bias && c + e < a.N ? a.bias[c + e] : 0.0f;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = t0 + j * 16 + row;
        if (t >= a.T) continue;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = acc[j][e] + bias[e];
        store_run<4>(a.Y, a.out, t, c, a.N, y);
    }
}

int64_t tiles(int64_t n, int b) { return (n + b - 1) / b; }
bool words_ok(const Mx4LinearArgs& a) { return a.nb % 4 == 0 && (((uintptr_t)a.a_scale | (uintptr_t)a.w_scale) & 3) == 0; }

// PER_CU: workgroups that a CU's LDS holds, each of which takes many tiles (0: one).
template <int BT, int BN, int WT, int WN, int ST, int PER_CU>
void run_tiles(Mx4LinearArgs a, hipStream_t stream)
{
    a.tiles_t = (int32_t)tiles(a.T, BT);
    a.tiles_n = (int32_t)tiles(a.N, BN);
    const int64_t all = (int64_t)a.tiles_t * a.tiles_n, most = (int64_t)device_cu_count() * PER_CU;
    const dim3 grid((unsigned)(PER_CU == 0 || all < most ? all : most)), block(WT * WN * 64);
    if (words_ok(a)) hipLaunchKernelGGL((tile_mx4_kernel<BT, BN, WT, WN, ST, true, (PER_CU > 0)>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((tile_mx4_kernel<BT, BN, WT, WN, 2, false, false>), dim3((unsigned)all), block, 0, stream, a);
}

template <int TT>
void run_few(const Mx4LinearArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)tiles(a.N, 16), (unsigned)tiles(a.T, TT * 16)), block(8 * 64);
    if (words_ok(a)) hipLaunchKernelGGL((few_mx4_kernel<TT, 8, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((few_mx4_kernel<TT, 8, false>), grid, block, 0, stream, a);
}

// Tiles as large as leave one for each CU: 256 x 256 reads least (1024 tiles of
// 8192 x 8192 270 us), and 128 x 128 in workgroups that take many hides the outputs of
// narrow products (360,000 x 768 to 128 channels: 48 us, with one tile a workgroup 66);
// with fewer tiles than CUs 64 x 64 (1024 x 4096 x 4096 in 256 tiles of 128 18.6 us, in
// 1024 of 64 23; 512 x 4096 x 4096 16.1 and 12.9; 4096 x 4096 x 4096 in tiles of 256 42
// and of 128 51). Where even tiles of 32 x 16 leave CUs idle, their waves split k (512 x
// 128 x 768 4.06 us against 4.16 in 64 x 64); with more of them than CUs the weights are
// read too often (48 x 4096 x 4096 12.5 against 8.1, 256 x 1024 x 1024 6.5 against 4.4).
void linear_once(const Mx4LinearArgs& a, hipStream_t stream)
{
    const int64_t cus = device_cu_count();
    if (a.T <= 16) run_few<1>(a, stream);
    else if (a.T <= 32 || tiles(a.T, 32) * tiles(a.N, 16) <= cus) run_few<2>(a, stream);
    else if (tiles(a.T, 256) * tiles(a.N, 256) >= cus && a.N > 128) run_tiles<256, 256, 2, 4, 2, 0>(a, stream);
    else if (tiles(a.T, 128) * tiles(a.N, 128) >= cus) run_tiles<128, 128, 2, 2, 2, 2>(a, stream);
    else run_tiles<64, 64, 2, 2, 4, 0>(a, stream);
}

}  // namespace

hipError_t launch_linear_mx4(Mx4LinearArgs a, hipStream_t stream)
{
    // One launch covers at most `step` rows, so that a grid's threads stay below
    // 2^32 (N is at most 2^26, so 256 rows make at most 2^22 tiles of 64 x 64); the
    // rows are independent.
    int64_t step = (int64_t)1 << 24;
    while (step > 256 && tiles(step, 64) * tiles(a.N, 64) > (1 << 22)) step /= 2;
    const int64_t es = a.out == kF32 ? 4 : 2;
    for (int64_t left = a.T; left > 0; left -= step) {
        a.T = left < step ? left : step;
        linear_once(a, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.A += step * a.nb * 16;
        a.a_scale += step * a.nb;
        a.Y = (char*)a.Y + step * a.N * es;
    }
    return hipSuccess;
}

}  // namespace maxsim
