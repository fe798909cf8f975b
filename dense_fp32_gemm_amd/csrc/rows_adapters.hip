// Low-rank adapters of many requests beside a shared product
// (include/gemm_f32_rows.h):  Y(t) = X(t).W + scale[a] (X(t).A_a).B_a.
//
// Few rows (the tiles of X.W would leave compute units idle), two launches:
//  1. step_kernel: X.W with K split over workgroups, and U = X(t).A_a, likewise,
//     as further workgroups of the same launch; binary32 partial sums to the workspace.
//  2. join_kernel: adds the parts in order and the row's U . B_a, vector FMAs.
// Many rows, three launches:
//  1. down_kernel: U = X(t).A_a, binary32 partial sums.
//  2. factor_kernel: adds the splits, scales, and writes each row of U as the
//     up-projection's operand: binary32 as it is, 16-bit types as high + low
//     parts (two 16-bit numbers per value: 16 to 22 bits instead of 8 to 11,
//     so that rounding U adds little to the rounding of Y) times a power of two
//     per row, which keeps them inside the type's range (see factor_kernel).
//  3. adapters_kernel: the tile of X.W, then for each adapter among its
//     rows the product of U's rows with B_a, of which only that adapter's rows
//     are added.
//
// An adapter's weights meet only its own rows' sums: infinities or NaN in one
// adapter do not reach other requests.

#include "rows_tile.h"

namespace rows {
namespace {

struct AdapterArgs {
    const void *X, *W, *A, *B;
    const int *adapter;
    const float *scale;
    void *Y;
    float *partial_u;    // [splits_u][T][R]
    float *partial_y;    // few rows: [splits][T][pitch]
    void *factor;        // many rows: [T][depth] elements
    float *unscale;      // many rows: [T]
    int64_t ldx, ldw, lda, ldb, ldy, stride_a, stride_b;
    int T, N, K, R, n;
    int splits_u, split_ku;  // down-projection: parts along K, k's of each
    int slots;               // waves that share a row tile's adapters
    int ranks;               // blocks of ranks
    int splits, split_k;     // few rows: parts of X.W along K
    int pitch;
    int depth;               // of factor's rows
    int tiles_m, tiles_n;
    int slots_big;           // many rows: workgroups the device holds at once
    int xcds;
    bool vector_y;           // Y's rows take stores of four elements
};

// Elements in a 128-byte panel row; rank indices such a panel of the up-projection
// holds: 16-bit panels are 64 deep, 32 high parts and then the low parts of the
// same ranks.
template <class E>
constexpr int panel_deep() { return 128 / E::kBytes; }
constexpr int kPanelRanks = 32;
template <class E>
int factor_depth(int R) { return (int)ceil_div(R, kPanelRanks) * panel_deep<E>(); }

// B_a's rows as the second operand of the up-projection: twice per panel for
// the 16-bit types.
template <class E, int RN, int NT>
struct UpRows : Across<E, RN, NT> {
    using Base = Across<E, RN, NT>;
    int R;
    __device__ inline UpRows(const typename E::T *base_, int tid_, int depth, int64_t ld_, int first_, int cols_, int R_)
        : Base(base_, tid_, depth, ld_, first_, cols_, R_), R(R_)
    {
    }
    __device__ inline int rank(int i, int k0) const { return k0 / Base::kDeep * kPanelRanks + this->krow(i) % kPanelRanks; }
    __device__ inline int64_t step() const { return kPanelRanks * this->ld; }
    __device__ inline bool last(int k0) const { return (k0 / Base::kDeep + 1) * kPanelRanks + E::kChunk >= R; }
    __device__ inline int left(int i, int k0) const { return rank(i, k0) < R ? Base::left(i, k0) : 0; }
    __device__ inline int inside(int i, int k0) const { return left(i, k0); }
    __device__ inline int64_t offset(int i, int) const
    {
        return this->krow(i) % kPanelRanks * this->ld + (int64_t)this->col(i) * E::kBytes;
    }
    static_assert(kPanelRanks % Base::kRowStep == 0, "a thread's rows wrap together");
    static __device__ inline int row_step(int i) { return i * Base::kRowStep % kPanelRanks; }
};

// The highest adapter number under `above` among a tile's rows, -1 if there is
// none.  which[q]: the adapter of row 64 * q + lane, -1: none.  The same in every lane and wave.
template <int WORDS>
__device__ inline int next_adapter(const int (&which)[WORDS], int above)
{
    uint32_t best = 0;                               // number + 1
#pragma unroll
    for (int q = 0; q < WORDS; ++q)
        best = max(best, which[q] < above ? (uint32_t)(which[q] + 1) : 0u);
    return (int)wave_max(best) - 1;
}

__device__ inline int adapter_of(const AdapterArgs &g, int64_t t, bool there)
{
    const int a = there ? g.adapter[t] : -1;
    return a >= 0 && a < g.n ? a : -1;
}

// ---------------------------------------------------------------------------
// Down-projection.  One wave: 16 rows, one part of K, RN ranks, and every
// slots-th adapter among the rows.  RN is 16, 32 or 64 (more ranks: further waves).
// ---------------------------------------------------------------------------
constexpr int kDownWaves = 4;
template <int RN>
constexpr int down_stages() { return RN == 16 ? 4 : RN == 32 ? 3 : 2; }
template <class E, int RN>
constexpr int down_lds() { return down_stages<RN>() * (16 + RN) * panel_deep<E>(); }   // elements of a wave

template <class E, int RN, bool DMA>
__device__ inline void down_item(const AdapterArgs &g, int64_t item, typename E::T *lds, int lane)
{
    using Ti = Tile<E, true, false, 16, RN, 1, 1>;
    using T = typename E::T;
    const int64_t tiles = (g.T + 15) / 16;
    if (item >= tiles * g.splits_u * g.slots * g.ranks)
        return;
    // neighbouring waves: the parts of K and the adapters of one row tile
    const int split = (int)(item % g.splits_u), slot = (int)(item / g.splits_u % g.slots);
    const int rank0 = (int)(item / ((int64_t)g.splits_u * g.slots) % g.ranks) * RN;
    const int t0 = (int)(item / ((int64_t)g.splits_u * g.slots * g.ranks)) * 16;
    const int k0 = split * g.split_ku, K = min(g.split_ku, g.K - k0);
    const int which[1] = {adapter_of(g, t0 + lane, lane < 16 && t0 + lane < g.T)};
    int nth = 0;
    for (int a = next_adapter(which, INT32_MAX); a >= 0; a = next_adapter(which, a)) {
        if (nth++ % g.slots != slot)
            continue;
        const uint64_t members = __ballot(which[0] == a);
        Ti tile;
        tile.clear();
        // Rows of other adapters come along; their sums are not stored.
        const Along<E, 16, kWave> x((const T *)g.X + t0 * g.ldx + k0, lane, K, g.ldx, g.T - t0,
                                    [&](int, int r) { return t0 + r < g.T ? r * g.ldx * E::kBytes : -1; });
        const Across<E, RN, kWave> w((const T *)g.A + a * g.stride_a + k0 * g.lda, lane, K, g.lda, rank0, g.R);
        group_sync<kWave>();
        sum_panels<E, DMA, down_stages<RN>(), false>(tile, K, x, w, lds, lane, 0, 0);
        tile.each(0, 0, lane, [&](int r, int c, f32x4 v) {
            if (members >> r & 1) {
                float *u = g.partial_u + ((int64_t)split * g.T + t0 + r) * g.R + rank0 + c;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rank0 + c + i < g.R)
                        u[i] = v[i];
            }
        });
    }
}

template <class E, int RN, bool DMA>
__global__ __launch_bounds__(kDownWaves *kWave) void down_kernel(AdapterArgs g)
{
    __shared__ __attribute__((aligned(16))) typename E::T lds[kDownWaves * down_lds<E, RN>()];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    down_item<E, RN, DMA>(g, (int64_t)blockIdx.x * kDownWaves + wave, lds + wave * down_lds<E, RN>(), threadIdx.x % kWave);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
constexpr int kStepBN = 64, kStepStages = 4;

// Workgroups 0 .. tiles_m * tiles_n * splits - 1: parts of X.W; then the down-projection.
// Bound by the weights' bytes: 32 rows of 32 requests, 4096 x 4096, R = 16, bf16:
// 13.5 us for the 34 MB of W and 4 MB of A (2.8 TB/s; about 3 us are the launch and the
// first panel's latency).
template <class E, int BM, int RN, bool DMA>
__global__ __launch_bounds__(kDownWaves *kWave) void step_kernel(AdapterArgs g)
{
    using T = typename E::T;
    constexpr int WM = BM == 16 ? 1 : 2, WN = 4 / WM, NT = kDownWaves * kWave;
    using Ti = Tile<E, true, false, BM, kStepBN, WM, WN>;
    constexpr int kTileLds = (DMA ? kStepStages : 2) * (Ti::kLdsA + Ti::kLdsB), kDownLds = kDownWaves * down_lds<E, RN>();
    __shared__ __attribute__((aligned(16))) T lds[kTileLds > kDownLds ? kTileLds : kDownLds];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int parts = g.tiles_m * g.tiles_n * g.splits;
    if ((int)blockIdx.x >= parts) {
        down_item<E, RN, DMA>(g, (int64_t)((int)blockIdx.x - parts) * kDownWaves + wave, lds + wave * down_lds<E, RN>(), lane);
        return;
    }
    const int wm = wave / WN, wn = wave % WN;
    const int tm = blockIdx.x % g.tiles_m, rest = blockIdx.x / g.tiles_m;   // rows share W's panels
    const int n0 = rest % g.tiles_n * kStepBN, split = rest / g.tiles_n;
    const int m0 = tm * BM, k0 = split * g.split_k, K = min(g.split_k, g.K - k0);
    Ti tile;
    tile.clear();
    const Along<E, BM, NT> x((const T *)g.X + m0 * g.ldx + k0, tid, K, g.ldx, g.T - m0,
                             [&](int, int r) { return m0 + r < g.T ? r * g.ldx * E::kBytes : -1; });
    const Across<E, kStepBN, NT> w((const T *)g.W + k0 * g.ldw, tid, K, g.ldw, n0, g.N);
    sum_panels<E, DMA, kStepStages, false>(tile, K, x, w, lds, tid, wm, wn);
    tile.each(wm, wn, lane, [&](int r, int c, f32x4 v) {
        // whole groups of four: rows of the parts are padded to a multiple of eight
        if (m0 + r < g.T && n0 + c < g.N)
            *reinterpret_cast<f32x4 *>(g.partial_y + ((int64_t)split * g.T + m0 + r) * g.pitch + n0 + c) = v;
    });
}

// One wave: a chunk per lane of one row's columns.  5.8 us for the same call: latency of
// the parts, then of U, then of B's rows.
template <class E>
__global__ __launch_bounds__(kWave) void join_kernel(AdapterArgs g)
{
    using T = typename E::T;
    __shared__ float u[GEMM_F32_MAX_RANK];
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.y;
    const int n = (blockIdx.x * kWave + lane) * E::kChunk;
    // The parts first: they wait for nothing.  kBatch parts' loads in flight.
    constexpr int kBatch = 8;
    float sum[E::kChunk] = {};
    auto add_parts = [&](int i0) {
        f32x4 v[kBatch][E::kChunk / 4];
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (int e = 0; e < E::kChunk / 4; ++e)
                v[q][e] = i0 + q < g.splits && n < g.N
                              ? *reinterpret_cast<const f32x4 *>(g.partial_y + ((int64_t)(i0 + q) * g.T + t) * g.pitch + n + 4 * e)
                              : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (int e = 0; e < E::kChunk; ++e)
                sum[e] += v[q][e / 4][e % 4];
    };
    const int a = g.R > 0 ? adapter_of(g, t, true) : -1;
    add_parts(0);
    for (int i = kBatch; i < g.splits; i += kBatch)
        add_parts(i);
    if (a >= 0) {
        const float s = g.scale != nullptr ? g.scale[a] : 1.f;
        for (int r = lane; r < g.R; r += kWave) {
            float part[kBatch], low = 0.f;
            for (int i0 = 0; i0 < g.splits_u; i0 += kBatch) {
#pragma unroll
                for (int q = 0; q < kBatch; ++q)
                    part[q] = i0 + q < g.splits_u ? g.partial_u[((int64_t)(i0 + q) * g.T + t) * g.R + r] : 0.f;
#pragma unroll
                for (int q = 0; q < kBatch; ++q)
                    low += part[q];
            }
            u[r] = s * low;
        }
    }
    __syncthreads();
    if (n >= g.N)
        return;
    if (a >= 0) {
        const T *B = (const T *)g.B + a * g.stride_b + n;
        for (int r0 = 0; r0 < g.R; r0 += kBatch) {   // kBatch rows of B in flight
            Chunk<E> b[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                b[q].raw = load_chunk<E, false>(B + (int64_t)(r0 + q) * g.ldb, r0 + q < g.R ? g.N - n : 0);
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                if (r0 + q < g.R)
#pragma unroll
                    for (int e = 0; e < E::kChunk; ++e)
                        sum[e] = fmaf(u[r0 + q], (float)b[q].e[e], sum[e]);
        }
    }
    Chunk<E> o;
#pragma unroll
    for (int e = 0; e < E::kChunk; ++e)
        o.e[e] = (T)sum[e];
    store_chunk<E, false>((T *)g.Y + t * g.ldy + n, o, g.N - n);
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------
// A wave per row.  2050 rows of rank 32: 5 us, latency of the parts.
//
// The scale of half rows puts the largest value next to the top of the type's range: a part
// has 11 bits down to 2^-14 and nothing under 2^-25, so the two together are off by at most
// 2^-22 of the value or 2^-39 of the row's largest.  (Sums of their products stay
// under 2^15 * 2^16 * 2 * 256.)  bfloat16 parts have binary32's range and 16 bits together; its
// rows are left alone but at the range's ends, where a low part would underflow or a high
// one round to infinity: scaled up to 1, a small row would overflow with large elements of B.
constexpr int kFactorThreads = 256;

template <class E>
__global__ __launch_bounds__(kFactorThreads) void factor_kernel(AdapterArgs g)
{
    using T = typename E::T;
    constexpr int kPer = GEMM_F32_MAX_RANK / kWave;  // ranks of a lane
    const int lane = threadIdx.x % kWave;
    const int64_t t = (int64_t)blockIdx.x * (kFactorThreads / kWave) + threadIdx.x / kWave;
    if (t >= g.T)
        return;
    const int a = adapter_of(g, t, true);
    if (a < 0)
        return;
    const float s = g.scale != nullptr ? g.scale[a] : 1.f;
    T *out = (T *)g.factor + t * g.depth;
    float u[kPer];
    float top = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int r = q * kWave + lane;
        u[q] = 0.f;
        if (r < g.R)
            for (int i = 0; i < g.splits_u; ++i)
                u[q] += g.partial_u[((int64_t)i * g.T + t) * g.R + r];
        u[q] = r < g.R ? u[q] * s : 0.f;             // what pads the ranks stays 0 under an infinite scale
        top = fmaxf(top, fabsf(u[q]) < INFINITY ? fabsf(u[q]) : 0.f);
    }
    if constexpr (E::kBytes == 4) {
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            if (q * kWave + lane < g.depth)
                out[q * kWave + lane] = u[q];
    } else {
#pragma unroll
        for (int d = kWave / 2; d > 0; d /= 2)
            top = fmaxf(top, __shfl_xor(top, d));
        // half: the row's largest finite value to [2^14, 2^15); bfloat16: to 2^-60 .. 2^101 if it
        // lies outside; rows without one as they are
        const int e = top > 0.f ? ilogbf(top) : 0;
        int up = e > 100 ? e - 100 : e < -60 ? e + 60 : 0;
        if (std::is_same<E, F16>::value && top > 0.f)
            up = max(e, -100) - 14;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int r = q * kWave + lane;
            const float x = ldexpf(u[q], -up);
            const T hi = (T)x;
            const float rest = x - (float)hi;
            if (r / 32 * 64 < g.depth) {
                out[r / 32 * 64 + r % 32] = hi;
                out[r / 32 * 64 + 32 + r % 32] = (T)(fabsf(rest) < INFINITY ? rest : 0.f);
            }
        }
        if (lane == 0)
            g.unscale[t] = ldexpf(1.f, up);
    }
}

// One tile of Y, rows from m0 on.  Bound by the panels' rate from L2 (about 16 bytes a clock and
// compute unit): 2050 x 4096 x 4096, R = 32, fp16: 87 us, 806 TFLOP/s, of which the low-rank
// addition is about 4; the library's bf16 product of 8192^3 runs at 1245.
template <class E, int BM, int BN, int WM, int WN, int S, bool DMA>
__device__ inline void adapters_tile(const AdapterArgs &g, int m0, int n0, typename E::T *lds)
{
    using Ti = Tile<E, true, false, BM, BN, WM, WN>;
    using T = typename E::T;
    constexpr int NT = Ti::kThreads;
    if (m0 >= g.T || n0 >= g.N)
        return;                                      // the whole workgroup
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / WN, wn = wave % WN;
    Ti tile;
    tile.clear();
    {
        const Along<E, BM, NT> x((const T *)g.X + m0 * g.ldx, tid, g.K, g.ldx, g.T - m0,
                                 [&](int, int r) { return m0 + r < g.T ? r * g.ldx * E::kBytes : -1; });
        const Across<E, BN, NT> w((const T *)g.W, tid, g.K, g.ldw, n0, g.N);
        sum_panels<E, DMA, S>(tile, g.K, x, w, lds, tid, wm, wn);
    }
    if (g.R > 0) {
        constexpr int kWords = (BM + kWave - 1) / kWave;
        int which[kWords], adds[Ti::kFm];            // adapters of the tile's rows; of those this lane adds to
        float unscale[Ti::kFm];
#pragma unroll
        for (int q = 0; q < kWords; ++q)
            which[q] = adapter_of(g, m0 + q * kWave + lane, q * kWave + lane < BM && m0 + q * kWave + lane < g.T);
#pragma unroll
        for (int m = 0; m < Ti::kFm; ++m) {
            const int r = wm * (BM / WM) + Ti::Fa::row_of(m, lane % 16);
            adds[m] = adapter_of(g, m0 + r, m0 + r < g.T);
            unscale[m] = E::kBytes == 2 && adds[m] >= 0 ? g.unscale[m0 + r] : 1.f;
        }
        static_assert(Ti::kSteps == 2 && (E::kBytes == 4 || Ti::kDeep == 2 * kPanelRanks), "a step for the high parts, one for the low");
        // Every row's U, whichever adapter made it (rows without one hold anything):
        // a row of sums is taken only with its own adapter's B.
        const Along<E, BM, NT> u((const T *)g.factor + (int64_t)m0 * g.depth, tid, g.depth, g.depth, g.T - m0,
                                 [&](int, int r) { return m0 + r < g.T ? (int64_t)r * g.depth * E::kBytes : -1; });
        for (int k0 = 0; k0 < g.depth; k0 += Ti::kDeep) {
            for (int a = next_adapter(which, INT32_MAX); a >= 0; a = next_adapter(which, a)) {
                const UpRows<E, BN, NT> b((const T *)g.B + a * g.stride_b, tid, g.depth, g.ldb, n0, g.N, g.R);
                __syncthreads();
                load_panel<E, DMA, NT>(u, k0, lds, tid);
                load_panel<E, DMA, NT>(b, k0, lds + Ti::kLdsA, tid);
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                __syncthreads();
                // The sums of one 16-row block at a time: a second set for the whole
                // tile would halve the waves a SIMD holds.
                typename Ti::Fb fb[Ti::kSteps];
#pragma unroll
                for (int step = 0; step < Ti::kSteps; ++step)
                    fb[step].read(lds + Ti::kLdsA, wn * (BN / WN), step, lane);
#pragma unroll
                for (int m = 0; m < Ti::kFm; ++m) {
                    Fragments<E, true, BM, 1> fa[Ti::kSteps];
#pragma unroll
                    for (int step = 0; step < Ti::kSteps; ++step)
                        fa[step].read(lds, wm * (BM / WM) + 16 * m, step, lane);
                    f32x4 add[Ti::kFn];
#pragma unroll
                    for (int n = 0; n < Ti::kFn; ++n) {
                        add[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int step = 0; step < Ti::kSteps; ++step) {
                            f32x4 sum = add[n];
#pragma unroll
                            for (int s = 0; s < kPerStep<E>; ++s)
                                sum = mfma<E>(fb[step].q[n], fa[step].q[0], sum, s);
                            // 16-bit types: step 0 holds the high parts, step 1 the low ones, which
                            // an infinity of B must not meet: their signs differ, or they are 0
                            if constexpr (E::kBytes == 2)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    sum[i] = step == 0 || fabsf(add[n][i]) < INFINITY ? sum[i] : add[n][i];
                            add[n] = sum;
                        }
                    }
                    const bool mine = adds[m] == a;
#pragma unroll
                    for (int n = 0; n < Ti::kFn; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)      // in place, nothing of the others' rows
                            tile.acc[m][n][i] = fmaf(unscale[m], mine ? add[n][i] : 0.f, tile.acc[m][n][i]);
                    __builtin_amdgcn_sched_barrier(0);   // one block's sums at a time in registers
                }
            }
        }
    }
    T *Y = (T *)g.Y;
    auto store = [&](auto vec) {
        tile.each(wm, wn, lane, [&](int r, int c, f32x4 v) {
            const int m = m0 + r, n = n0 + c;
            if (m < g.T && n < g.N)
                store4<E, decltype(vec)::value>(Y + m * g.ldy + n, v, g.N - n);
        });
    };
    if (g.vector_y)
        store(std::true_type{});
    else
        store(std::false_type{});
}

// The tiles of many rows.  16-bit types: BM x 256 (see many_rows()), one workgroup
// a compute unit; 256 x 256 tiles cut the last round.  binary32, bound by the matrix
// cores: 64 x 64.
template <class E, int BM>
struct Big {
    static constexpr int BN = E::kBytes == 2 ? 256 : 64, WM = 2, WN = E::kBytes == 2 ? 4 : 2;
    static constexpr int kThreads = WM * WN * kWave;
    static constexpr bool kCut = BM == 256;
    static constexpr int S = BM == 160 ? 3 : 2;                              // panels in LDS
    static constexpr int kLds = (kCut ? 9 * 128 : S * (BM + BN)) * panel_deep<E>();   // cut: three of a half, four of a quarter
};

template <class E, int BM, bool DMA>
__global__ __launch_bounds__((Big<E, BM>::kThreads), 2) void adapters_kernel(AdapterArgs g)
{
    using B = Big<E, BM>;
    __shared__ __attribute__((aligned(16))) typename E::T lds[B::kLds];
    const int total = g.tiles_m * g.tiles_n;
    if constexpr (!B::kCut) {
        const int t = die_contiguous(blockIdx.x, total, g.xcds);
        adapters_tile<E, BM, B::BN, B::WM, B::WN, B::S, DMA>(g, t % g.tiles_m * BM, t / g.tiles_m * B::BN, lds);
    } else {
        constexpr int H = BM / 2, BN = B::BN;
        const Part part = part_of(blockIdx.x, total, g.slots_big, g.xcds);
        if (part.tile < 0)
            return;
        const int m0 = part.tile % g.tiles_m * BM, n0 = part.tile / g.tiles_m * BN;
        if (part.cut == 1)
            adapters_tile<E, BM, BN, B::WM, B::WN, 2, DMA>(g, m0, n0, lds);
        else if (part.cut == 2)
            adapters_tile<E, H, BN, B::WM, B::WN, 3, DMA>(g, m0 + part.piece * H, n0, lds);
        else
            adapters_tile<E, H, BN / 2, B::WM, B::WN, 4, DMA>(g, m0 + part.piece % 2 * H, n0 + part.piece / 2 * (BN / 2), lds);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// How a call is split; sized for 256 compute units whatever the device, so
// that the workspace depends on the arguments alone.
struct Split {
    bool few;
    int splits, split_k;                             // X.W, few rows
    int splits_u, split_ku, slots, ranks, rank_block;
    int pitch, depth;
    size_t partial_y, factor, unscale, bytes;        // workspace offsets
};

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// Parts of `panels` panels: `want` of them, none under `least` panels.
void cut(int64_t panels, int64_t want, int64_t least, int panel, int *parts, int *length)
{
    int64_t s = want < panels / least ? want : panels / least;
    if (s < 1)
        s = 1;
    const int64_t each = panels > 0 ? ceil_div(panels, s) : 0;
    *parts = panels > 0 ? (int)ceil_div(panels, each) : 1;
    *length = (int)(each * panel);
}

// Few rows: fewer than 128 tiles of 128 x 128, and no more rows than the parts' own traffic and
// join_kernel's reads of B_a, once a row, allow: few_rows().
// Ranks: many rows of 17 to 32 take a block of 32 of them (2050 rows, R = 32: 105 against
// 108 with 64; 8192 rows, K = N = 1024: 45 against 47).
//
// us a call in a graph, 8 adapters, rows side by side, few against many:
//   bfloat16, K = N = 1024, R = 16: 512 rows 18 and 24, 1024: 21 and 24, 2048: 27 and 25;
//     R = 32: 512 rows 24 and 26, 1024: 28 and 25; R = 64: 640 rows 29 and 33, 1024: 31 and 28;
//     R = 128: 320 rows 32 and 49, 512: 38 and 35; R = 256: 384 rows 54 and 72, 512: 56 and 50,
//     2048: 99 and 42;
//   K = N = 2048, R = 64: 512 rows 37 and 40; R = 32: 768 rows 44 and 37;
//   K = N = 4096, 384 rows: R = 16 48 and 53, R = 64 63 and 61, R = 256 107 and 101;
//   binary32, K = N = 1024, R = 16: 512 rows 27 and 34; R = 64: 320 rows 37 and 45, 512: 40 and 40;
//     R = 128: 256 rows 46 and 46, 320: 62 and 54; R = 256: 256 rows 67 and 64, 512: 75 and 57;
//   K = N = 2048, 512 rows: R = 16 57 and 58, R = 32 72 and 59; K = N = 4096, 384 rows: R = 16 134
//   and 143, R = 32 141 and 146, R = 64 148 and 152, R = 128 239 and 165.
// Narrow outputs of more rows gain nothing (bfloat16, K = 8192, N = 64, R = 16: 4096 rows 85 and 86).
template <class E>
int few_rows(int R)
{
    if (E::kBytes == 4)
        return R <= 16 ? 512 : R <= 64 ? 320 : 256;
    return R <= 16 ? 2048 : R <= 64 ? 640 : 384;
}

template <class E>
Split plan(int T, int N, int K, int R)
{
    Split p{};
    const int panel = panel_deep<E>();
    const int64_t panels = ceil_div(K, panel), rows16 = ceil_div(T, 16);
    p.few = ceil_div(T, 128) * ceil_div(N, 128) < 128 && T <= few_rows<E>(R);
    p.rank_block = R <= 16 ? 16 : R <= 32 && !p.few ? 32 : 64;
    p.ranks = (int)ceil_div(R, p.rank_block);
    if (R > 0) {
        // about a thousand waves: up to 16 for the adapters of a row tile when rows are few
        p.slots = p.few ? (T < 16 ? T : 16) : 1;
        cut(panels, 1024 / (rows16 * p.slots * p.ranks), 4, panel, &p.splits_u, &p.split_ku);
    }
    if (p.few) {
        const int64_t tiles = ceil_div(T, T <= 16 ? 16 : 64) * ceil_div(N, kStepBN);
        cut(panels, 512 / tiles, 4, panel, &p.splits, &p.split_k);
        p.pitch = (int)ceil_div(N, 8) * 8;
    }
    p.depth = factor_depth<E>(R);
    size_t at = round16((size_t)p.splits_u * (size_t)T * (size_t)R * 4);
    p.partial_y = at;
    if (p.few) {
        at += round16((size_t)p.splits * (size_t)T * (size_t)p.pitch * 4);
    } else if (R > 0) {
        p.factor = at;
        at += round16((size_t)T * (size_t)p.depth * E::kBytes);
        p.unscale = at;
        at += round16((size_t)T * 4);
    }
    p.bytes = at;
    return p;
}

// A grid has fewer than 2^32 threads, and there is a wave per token.
constexpr int kMaxTokens = 1 << 25;
// Most rows of an operand that one panel's offsets span (a tile's, or a panel's depth).
constexpr int kPanelRows = 256;

bool short_ld(int64_t ld, int cols) { return ld < at_least_one(cols); }

template <class E, int RN>
int64_t down_blocks(const AdapterArgs &g)
{
    return ceil_div(ceil_div(g.T, 16) * g.splits_u * g.slots * g.ranks, kDownWaves);
}

template <class E, int RN>
int run_few(AdapterArgs g, bool low, bool dma, hipStream_t stream)
{
    const int64_t down = low ? down_blocks<E, RN>(g) : 0;
    auto launch = [&](auto bm, auto direct) {
        constexpr int BM = decltype(bm)::value;
        g.tiles_m = (int)ceil_div(g.T, BM);
        g.tiles_n = (int)ceil_div(g.N, kStepBN);
        const int64_t grid = (int64_t)g.tiles_m * g.tiles_n * g.splits + down;
        step_kernel<E, BM, RN, decltype(direct)::value><<<(unsigned)grid, kDownWaves * kWave, 0, stream>>>(g);
    };
    if (g.T <= 16 && dma)
        launch(std::integral_constant<int, 16>{}, std::true_type{});
    else if (g.T <= 16)
        launch(std::integral_constant<int, 16>{}, std::false_type{});
    else if (dma)
        launch(std::integral_constant<int, 64>{}, std::true_type{});
    else
        launch(std::integral_constant<int, 64>{}, std::false_type{});
    const dim3 grid((unsigned)ceil_div(g.N, kWave * E::kChunk), (unsigned)g.T);
    join_kernel<E><<<grid, kWave, 0, stream>>>(g);
    return launched();
}

template <class E, int BM>
int launch_many(AdapterArgs g, bool dma, hipStream_t stream)
{
    using B = Big<E, BM>;
    const int64_t tm = ceil_div(g.T, BM), tn = ceil_div(g.N, B::BN);
    g.slots_big = (int)gemm_f32_internal::current_device().cus;
    // cutting the last round adds at most three pieces for a quarter of the slots
    const int64_t grid = tm * tn + (B::kCut ? g.slots_big : 0);
    if (grid > (int64_t)UINT32_MAX / B::kThreads)
        return GEMM_F32_ERR_DIM;
    g.tiles_m = (int)tm;
    g.tiles_n = (int)tn;
    if (dma)
        adapters_kernel<E, BM, true><<<(unsigned)grid, B::kThreads, 0, stream>>>(g);
    else
        adapters_kernel<E, BM, false><<<(unsigned)grid, B::kThreads, 0, stream>>>(g);
    return launched();
}

// The tile: its panels' rate from L2 bounds a compute unit, so the cost of a round is about
// BM + 256.  256 x 256, whose last round is cut into halves or quarters, but 160 x
// 256 where those fit one round and the halves of the others do not (bf16, K = N = 4096, R =
// 16, us a call, 256 against 160: 1024 rows 64 and 93, 2050: 125 and 95, 2560:
// 123 and 97, 2600: 124 and 155, 8192: 274 and 324).  binary32: 64 x 64.
template <class E>
int many_rows(const AdapterArgs &g, bool dma, hipStream_t stream)
{
    if constexpr (E::kBytes == 4) {
        return launch_many<E, 64>(g, dma, stream);
    } else {
        const int64_t cus = gemm_f32_internal::current_device().cus, tn = ceil_div(g.N, 256);
        if (2 * ceil_div(g.T, 256) * tn > cus && ceil_div(g.T, 160) * tn <= cus)
            return launch_many<E, 160>(g, dma, stream);
        return launch_many<E, 256>(g, dma, stream);
    }
}

template <class E, int RN>
int run_many(const AdapterArgs &g, bool low, bool dma, bool dma_down, hipStream_t stream)
{
    if (low) {
        const int64_t blocks = down_blocks<E, RN>(g);
        if (dma_down)
            down_kernel<E, RN, true><<<(unsigned)blocks, kDownWaves * kWave, 0, stream>>>(g);
        else
            down_kernel<E, RN, false><<<(unsigned)blocks, kDownWaves * kWave, 0, stream>>>(g);
        factor_kernel<E><<<(unsigned)ceil_div(g.T, kFactorThreads / kWave), kFactorThreads, 0, stream>>>(g);
    }
    return many_rows<E>(g, dma, stream);
}

}  // namespace
}  // namespace rows

using namespace rows;

extern "C" {

size_t gemm_f32_adapters_ws_size(int type, int T, int N, int K, int R)
{
    if (T <= 0 || T > kMaxTokens || N == 0 || bad_size(N) || bad_size(K) || R < 0 || R > GEMM_F32_MAX_RANK)
        return 0;
    size_t bytes = 0;
    with_type(type, [&](auto e) { bytes = plan<decltype(e)>(T, N, K, R).bytes; });
    return bytes;
}

int gemm_f32_adapters(int type, int T, int N, int K, int R, int n, const void *X, int ldx, const void *W, int ldw,
                      const void *A, int lda, int64_t stride_a, const void *B, int ldb, int64_t stride_b,
                      const int *adapter, const float *scale, void *Y, int ldy, void *ws, size_t ws_bytes,
                      hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (T < 0 || T > kMaxTokens || bad_size(N) || bad_size(K) || R < 0 || R > GEMM_F32_MAX_RANK || n < 0)
        return GEMM_F32_ERR_DIM;
    const int64_t tile = type == GEMM_F32_TYPE_F32 ? 64 : 256, threads = type == GEMM_F32_TYPE_F32 ? 256 : 512;
    if (ceil_div(T, tile) * ceil_div(N, tile) > UINT32_MAX / threads - 1024)
        return GEMM_F32_ERR_DIM;                     // a grid has fewer than 2^32 threads
    if (short_ld(ldx, K) || short_ld(ldw, N) || short_ld(ldy, N) || short_ld(lda, R) || short_ld(ldb, N) ||
        (n > 1 && (stride_a < K * (int64_t)lda || stride_b < R * (int64_t)ldb)))
        return GEMM_F32_ERR_LD;
    if (T == 0 || N == 0)
        return GEMM_F32_OK;
    const bool low = R > 0 && n > 0;
    if (Y == nullptr || (K > 0 && (X == nullptr || W == nullptr)) ||
        (low && (B == nullptr || adapter == nullptr || (K > 0 && A == nullptr))))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(X, b) || !aligned_to(W, b) || !aligned_to(Y, b) ||
        (low && (!aligned_to(A, b) || !aligned_to(B, b) || !aligned_to(adapter, 4) || !aligned_to(scale, 4))))
        return GEMM_F32_ERR_ALIGN;
    const size_t need = gemm_f32_adapters_ws_size(type, T, N, K, R);
    if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned_to(ws, 16)))
        return GEMM_F32_ERR_WORKSPACE;

    const bool dma_x = dma_rows(type, X, ldx, kPanelRows), dma_w = dma_rows(type, W, ldw, kPanelRows);
    const bool dma_a = !low || (dma_rows(type, A, lda, kPanelRows) && (n == 1 || stride_a * b % 4 == 0));
    const bool dma_b = !low || (dma_rows(type, B, ldb, kPanelRows) && (n == 1 || stride_b * b % 4 == 0));
    int rc = GEMM_F32_OK;
    with_type(type, [&](auto e) {
        using E = decltype(e);
        const Split p = plan<E>(T, N, K, R);
        AdapterArgs g{};
        g.X = X, g.W = W, g.A = A, g.B = B, g.Y = Y;
        g.adapter = adapter, g.scale = scale;
        g.partial_u = (float *)ws;
        g.partial_y = (float *)((char *)ws + p.partial_y);
        g.factor = (char *)ws + p.factor;
        g.unscale = (float *)((char *)ws + p.unscale);
        g.ldx = ldx, g.ldw = ldw, g.lda = lda, g.ldb = ldb, g.ldy = ldy;
        g.stride_a = stride_a, g.stride_b = stride_b;
        g.T = T, g.N = N, g.K = K, g.R = low ? R : 0, g.n = n;
        g.splits_u = p.splits_u, g.split_ku = p.split_ku, g.slots = p.slots, g.ranks = p.ranks;
        g.splits = p.splits, g.split_k = p.split_k;
        g.pitch = p.pitch, g.depth = p.depth;
        g.xcds = gemm_f32_internal::current_device().xcds;
        g.vector_y = vector_rows(type, Y, ldy, 0, N);
        if (p.few && p.rank_block == 16)
            rc = run_few<E, 16>(g, low, dma_x && dma_w && dma_a, stream);
        else if (p.few)
            rc = run_few<E, 64>(g, low, dma_x && dma_w && dma_a, stream);
        else if (p.rank_block == 32)
            rc = run_many<E, 32>(g, low, dma_x && dma_w && dma_b, dma_x && dma_a, stream);
        else if (p.rank_block == 16)
            rc = run_many<E, 16>(g, low, dma_x && dma_w && dma_b, dma_x && dma_a, stream);
        else
            rc = run_many<E, 64>(g, low, dma_x && dma_w && dma_b, dma_x && dma_a, stream);
    });
    return rc;
}

}  // extern "C"
