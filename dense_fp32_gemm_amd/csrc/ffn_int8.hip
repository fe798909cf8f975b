// The product of 8-bit rows and 8-bit weights with a scale for each token and channel
// (include/gemm_f32_ffn.h).
//
//  * few rows: int8_few_kernel.  16 channels a workgroup, K over its waves,
//    operands straight into registers.  Bound by the weights' bytes and one load's way: 4096 x 4096, weights from
//    memory, in a graph: one row 5.9 us, 16 rows 7.4; 8192 x 8192, one row 15.2 us, 4.4 TB/s.
//  * else int8_kernel: tiles as in rows_tile.h, both operands' k contiguous.  8192 x 4096, K = 4096: 117 us, 2350 TOP/s;
//    8192 x 8192, K = 8192: 431 us, 2550 TOP/s (the library's 8-bit product without scales 127 and 517).  Bound by the card's
//    power and the sums' loop: 11 us a round of tiles and 1024 k; 14 us a round for its start and its stores.

#include "ffn_gate.h"
#include "rows_groups.h"

namespace ffn {
namespace {

struct Int8Args {
    const int8_t *Q, *W;
    const float *scale, *w_scale, *bias;
    void *Y;
    int64_t ldq, ldw, ldy;
    int T, N, K;
    int tiles_m, tiles_n, slots, xcds;
    bool vector_y;
};

// Scales (and biases) of four neighbouring channels from n on.
struct Channels {
    f32x4 scale, bias;
    __device__ inline void load(const Int8Args &g, int n)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = n + i < g.N ? n + i : g.N - 1;
            scale[i] = g.w_scale[c];
            bias[i] = g.bias != nullptr ? g.bias[c] : 0.f;
        }
    }
    // Their sums of a row whose scale is s.  Binary32 results are rounded once, from binary64, where the scales' product is
    // exact (4096 channels, K = 4096: 8192 rows 119 us, 120 with binary32's three roundings; 512 rows 16.6 and 16.3); for
    // the 16-bit types each of those is little beside theirs (2^-13 of it for half, 2^-16 for bf16).
    template <class Out>
    __device__ inline f32x4 scaled(i32x4 v, float s) const
    {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Out::kBytes == 4)
                y[i] = (float)fma((double)v[i], (double)s * (double)scale[i], (double)bias[i]);
            else
                y[i] = (float)v[i] * (s * scale[i]) + bias[i];
        }
        return y;
    }
};

template <class Out, bool VEC>
__device__ inline void int8_store(const Int8Args &g, int64_t t, int n, f32x4 y)
{
    store4<Out, VEC>((typename Out::T *)g.Y + t * g.ldy + n, y, g.N - n);
}

template <class Out, int BM, int BN, int WM, int WN, int S, bool DMA>
__device__ inline void int8_tile(const Int8Args &g, int m0, int n0, int8_t *lds)
{
    using Ti = Tile<I8, true, true, BM, BN, WM, WN>;
    constexpr int NT = Ti::kThreads;
    if (m0 >= g.T || n0 >= g.N)
        return;                                      // the whole workgroup
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / WN, wn = wave % WN;
    Ti tile;
    tile.clear();
    const Along<I8, BM, NT> a(g.Q + m0 * g.ldq, tid, g.K, g.ldq, g.T - m0,
                              [&](int, int r) { return m0 + r < g.T ? r * g.ldq : -1; });
    const Along<I8, BN, NT> b(g.W + n0 * g.ldw, tid, g.K, g.ldw, g.N - n0,
                              [&](int, int r) { return n0 + r < g.N ? r * g.ldw : -1; });
    sum_panels<I8, DMA, S>(tile, g.K, a, b, lds, tid, wm, wn);
    // All scales, then their use (8192 x 4096, K = 4096: loaded one by one between the stores 171 us against 154); wide and
    // narrow stores apart (merged, the compiler makes 2- and 4-byte pieces of the wide ones: 154 against 117).
    const int i = lane % 16, h = lane / 16, row = m0 + wm * (BM / WM) + i, col = n0 + wn * (BN / WN) + 4 * h;
    float scale[Ti::kFm];
    Channels channels[Ti::kFn];
#pragma unroll
    for (int m = 0; m < Ti::kFm; ++m)
        scale[m] = g.scale[min(row + 16 * m, g.T - 1)];
#pragma unroll
    for (int n = 0; n < Ti::kFn; ++n)
        channels[n].load(g, col + 16 * n);
    auto store = [&](auto vec) {
#pragma unroll
        for (int m = 0; m < Ti::kFm; ++m)
#pragma unroll
            for (int n = 0; n < Ti::kFn; ++n)
                if (row + 16 * m < g.T && col + 16 * n < g.N)
                    int8_store<Out, decltype(vec)::value>(g, row + 16 * m, col + 16 * n, channels[n].template scaled<Out>(tile.acc[m][n], scale[m]));
    };
    if (g.vector_y)
        store(std::true_type{});
    else
        store(std::false_type{});
}

// Tiles are numbered in bands as those of a group (see kBand; 8192 x 4096, K = 4096: 165 us, whole columns 171).
template <class Out, int BM, int BN, int WM, int WN, int S, bool CUT, bool DMA>
__global__ __launch_bounds__(WM *WN *kWave, 2) void int8_kernel(Int8Args g)
{
    constexpr int kPanel = (BM + BN) * kDeep16 * I8::kChunk;
    // (S = 2) two panels of the whole tile, three of a half, four of a quarter
    __shared__ __attribute__((aligned(16))) int8_t lds[CUT && DMA ? 9 * kPanel / 4 : (DMA ? S : 2) * kPanel];
    static_assert(!CUT || (S == 2 && BM == BN), "panels of cut tiles");
    const int total = g.tiles_m * g.tiles_n;
    Part part{-1, 1, 0};
    if constexpr (CUT)
        part = part_of(blockIdx.x, total, g.slots, g.xcds);
    else if ((int)blockIdx.x < total)
        part.tile = die_contiguous(blockIdx.x, total, g.xcds);
    if (part.tile < 0)
        return;                                      // the whole workgroup
    const int from = part.tile / (kBand * g.tiles_n) * kBand, q = part.tile - from * g.tiles_n, high = min(kBand, g.tiles_m - from);
    const int m0 = (from + q % high) * BM, n0 = q / high * BN;
    if (!CUT || part.cut == 1)
        int8_tile<Out, BM, BN, WM, WN, S, DMA>(g, m0, n0, lds);
    if constexpr (CUT) {
        if (part.cut == 2)
            int8_tile<Out, BM / 2, BN, WM, WN, 3, DMA>(g, m0 + part.piece * (BM / 2), n0, lds);
        else if (part.cut == 4)
            int8_tile<Out, BM / 2, BN / 2, WM, WN, 4, DMA>(g, m0 + part.piece % 2 * (BM / 2), n0 + part.piece / 2 * (BN / 2), lds);
    }
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;                         // of a workgroup

// 16 channels and up to 16 MT rows a workgroup.  Wave w takes every kFewWaves-th block of 64 STEPS
// k: 16 bytes a lane, 64 bytes of a row side by side a step, all steps' loads before the first product.  The waves'
// sums meet in LDS.
template <class Out, bool VEC, int MT, int STEPS>
__global__ __launch_bounds__(kFewWaves *kWave) void int8_few_kernel(Int8Args g)
{
    constexpr int kBlock = STEPS * 64;
    __shared__ i32x4 part[kFewWaves][MT][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, i = lane % 16, h = lane / 16;
    const int n0 = blockIdx.x * 16;
    const bool channel = n0 + i < g.N;
    const int8_t *w = g.W + (channel ? n0 + i : 0) * g.ldw;
    i32x4 acc[MT] = {};
    for (int k0 = wave * kBlock; k0 < g.K; k0 += kFewWaves * kBlock) {
        u32x4 b[STEPS], a[MT][STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + 64 * s + 16 * h, left = g.K - k;
            b[s] = load_chunk<I8, VEC>(w + k, channel ? left : 0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int t = 16 * m + i;
                a[m][s] = load_chunk<I8, VEC>(g.Q + (t < g.T ? t : 0) * g.ldq + k, t < g.T ? left : 0);
            }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m] = mfma<I8>(b[s], a[m][s], acc[m], 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
        part[wave][m][lane] = acc[m];
    __syncthreads();
    for (int m = wave; m < MT; m += kFewWaves) {
        const int t = 16 * m + i, n = n0 + 4 * h;
        Channels channels;
        channels.load(g, n);
        const float s = g.scale[min(t, g.T - 1)];
        i32x4 sum = part[0][m][lane];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v)
            sum += part[v][m][lane];
        if (t < g.T && n < g.N)
            int8_store<Out, false>(g, t, n, channels.template scaled<Out>(sum, s));
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <class Out, int BM, int BN, int WM, int WN, int S, int PER_CU>
int launch_int8(Int8Args g, bool dma, hipStream_t stream, bool go)
{
    const int64_t tiles_m = ceil_div(g.T, BM), tiles_n = ceil_div(g.N, BN);
    g.slots = (int)gemm_f32_internal::current_device().cus * PER_CU;
    // cutting the last round adds at most three pieces for a quarter of the slots
    const int64_t grid = tiles_m * tiles_n + g.slots;
    if (grid > kMaxTiles)
        return GEMM_F32_ERR_DIM;
    if (!go || tiles_m * tiles_n == 0)
        return GEMM_F32_OK;
    g.tiles_m = (int)tiles_m;
    g.tiles_n = (int)tiles_n;
    constexpr bool kCut = PER_CU > 0;
    if (dma)
        int8_kernel<Out, BM, BN, WM, WN, S, kCut, true><<<(int)grid, WM * WN * kWave, 0, stream>>>(g);
    else
        int8_kernel<Out, BM, BN, WM, WN, S, kCut, false><<<(int)grid, WM * WN * kWave, 0, stream>>>(g);
    return launched();
}

// Rows of the few-row kernel.  Every workgroup reads all rows, which the caches bear up to one workgroup a
// compute unit (us in a graph, weights from HBM, against 32 x 64 tiles: 4096 channels, K = 4096: 16 rows 7.4 and 11.8, 32
// rows 10.0 and 12.0, 48 rows 12.0 and 11.9; 2048 channels, K = 8192: 32 rows 15.1 and 20.0, 48 rows 19.4 and 19.7;
// 8192 channels, K = 8192: 16 rows 19.6 and 21.2, 32 rows 28.0 and 21.7).
int few_rows(int N) { return ceil_div(N, 16) <= gemm_f32_internal::current_device().cus ? 48 : 16; }

// The largest tile of which there is one for every compute unit (us, all at 4096 channels, K = 4096: 128 rows 11.7 with
// 32 x 64, 13.0 with 64 x 64, 15.6 with 64 x 128; 256 rows 14.0, 13.7, 15.9; 512 rows 26.0, 18.5, 17.0).
// 256 x 256 tiles from a quarter of the units on, because they are cut there (1024 rows 26.2 against 25.9 for
// 64 x 128, 1536 rows 34.4 against 43.1, 2048 rows 37.8 against 49.9).  That branch does not look at the rows: with
// 16640 channels or more it takes 17 to 255 rows too, mostly padding (28672 channels, K = 4096: 17 rows 34.4 us, 64 37.2,
// 128 41.2, whose weights alone are 25 at a copy's rate).
int launch_int8(int type, const Int8Args &g, bool dma, bool vec, hipStream_t stream, bool go)
{
    int rc = GEMM_F32_OK;
    const int64_t cus = gemm_f32_internal::current_device().cus;
    auto tiles = [&](int bm, int bn) { return ceil_div(g.T, bm) * ceil_div(g.N, bn); };
    with_type(type, [&](auto e) {
        using Out = decltype(e);
        if (g.T <= few_rows(g.N)) {
            const int64_t grid = ceil_div(g.N, 16);
            if (grid > kMaxTiles) {
                rc = GEMM_F32_ERR_DIM;
                return;
            }
            if (!go || g.T == 0 || grid == 0)
                return;
            auto few = [&](auto mt, auto steps) {
                constexpr int MT = decltype(mt)::value, STEPS = decltype(steps)::value;
                if (vec)
                    int8_few_kernel<Out, true, MT, STEPS><<<(int)grid, kFewWaves * kWave, 0, stream>>>(g);
                else
                    int8_few_kernel<Out, false, MT, STEPS><<<(int)grid, kFewWaves * kWave, 0, stream>>>(g);
            };
            using std::integral_constant;
            if (g.T <= 16)
                few(integral_constant<int, 1>{}, integral_constant<int, 8>{});
            else if (g.T <= 32)
                few(integral_constant<int, 2>{}, integral_constant<int, 4>{});
            else
                few(integral_constant<int, 3>{}, integral_constant<int, 4>{});
            rc = launched();
        } else if (4 * tiles(256, 256) > cus) {
            rc = launch_int8<Out, 256, 256, 2, 4, 2, 1>(g, dma, stream, go);
        } else if (tiles(64, 128) >= cus) {
            rc = launch_int8<Out, 64, 128, 2, 2, 3, 0>(g, dma, stream, go);
        } else if (tiles(64, 64) >= cus) {
            rc = launch_int8<Out, 64, 64, 2, 2, 4, 0>(g, dma, stream, go);
        } else {
            rc = launch_int8<Out, 32, 64, 1, 4, 4, 0>(g, dma, stream, go);
        }
    });
    return rc;
}

// Rows of 8-bit elements that the direct loads can address (see dma_rows()).
bool dma_bytes(const void *p, int64_t ld) { return aligned_to(p, 4) && ld % 4 == 0 && kPanelRows * ld < (int64_t)kNowhere - 16; }
bool chunk_bytes(const void *p, int64_t ld, int K) { return aligned_to(p, 16) && ld % 16 == 0 && K % 16 == 0; }

}  // namespace
}  // namespace ffn

using namespace ffn;

extern "C" int gemm_f32_int8(int type, int T, int N, int K, const int8_t *Q, int ldq, const float *scale, const int8_t *W,
                             int ldw, const float *w_scale, const float *bias, void *Y, int ldy, hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (bad_size(T) || bad_size(N) || K < 0 || K > GEMM_F32_MAX_INT8_DEPTH)
        return GEMM_F32_ERR_DIM;
    const Int8Args g{Q, W, scale, w_scale, bias, Y, ldq, ldw, ldy, T, N, K, 0, 0, 0, gemm_f32_internal::current_device().xcds,
                     vector_rows(type, Y, ldy, 0, N)};
    const int rc = launch_int8(type, g, false, false, nullptr, false);
    if (rc != GEMM_F32_OK)
        return rc;
    if (short_ld(ldq, K) || short_ld(ldw, K) || short_ld(ldy, N))
        return GEMM_F32_ERR_LD;
    if (T == 0 || N == 0)
        return GEMM_F32_OK;
    if ((K > 0 && (Q == nullptr || W == nullptr)) || scale == nullptr || w_scale == nullptr || Y == nullptr)
        return GEMM_F32_ERR_NULL;
    if (!aligned_to(scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(bias, 4) || !aligned_to(Y, type_bytes(type)))
        return GEMM_F32_ERR_ALIGN;
    return launch_int8(type, g, dma_bytes(Q, ldq) && dma_bytes(W, ldw), chunk_bytes(Q, ldq, K) && chunk_bytes(W, ldw, K),
                       stream, true);
}
