// Low-rank adapters of many requests beside a shared product
// (include/gemm_f32_rows.h):  Y(t) = X(t).W + scale[a] (X(t).A_a).B_a.
//
//  1. down_kernel: U = X(t).A_a, 16 rows of X a wave, the K sum split over
//     workgroups; binary32 partial sums to the workspace.
//  2. factor_kernel: adds the splits, scales, and writes each row of U as the
//     up-projection's operand: binary32 as it is, 16-bit types as high + low
//     parts (two 16-bit numbers per value: 16 to 22 bits instead of 8 to 11,
//     so that rounding U adds nothing to the rounding of Y) times a power of two
//     per row, which keeps them inside the type's range.
//  3. adapters_kernel: the tile of X.W, then for each adapter among its
//     rows the product of U's rows with B_a into a second set of sums,
//     of which only that adapter's rows are added.
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
    float *partial;      // [splits][T][R]
    void *factor;        // [T][depth] elements
    float *unscale;      // [T]
    int64_t ldx, ldw, lda, ldb, ldy, stride_a, stride_b;
    int T, N, K, R, n;
    int splits, split_k; // down-projection: workgroups along K, k's of each
    int depth;           // of factor's rows
    int tiles_m, tiles_n;
    int xcds;
    bool vector_y;       // Y's rows take stores of four elements
};

// Rank indices a panel of the up-projection holds: 16-bit panels are 64 deep,
// 32 high parts and then the 32 low parts of the same ranks.
template <class E>
constexpr int panel_deep() { return 128 / E::kBytes; }
template <class E>
int factor_depth(int R) { return (int)ceil_div(R, 32) * panel_deep<E>(); }

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
    __device__ inline int rank(int i, int k0) const { return k0 / panel_deep<E>() * 32 + this->krow(i) % 32; }
    __device__ inline int64_t step() const { return 32 * this->ld; }
    __device__ inline bool partial(int k0) const { return (k0 / panel_deep<E>() + 1) * 32 > R; }
    __device__ inline int left(int i, int k0) const { return rank(i, k0) < R ? Base::left(i, k0) : 0; }
    __device__ inline int64_t offset(int i, int) const
    {
        return this->krow(i) % 32 * this->ld + (int64_t)this->col(i) * E::kBytes;
    }
};

// Calls f(a, members) for each adapter a among up to 128 rows, members being
// bit masks of its rows.  which: the adapter of row `lane` and of row 64 + lane, -1:
// none.  The same in every wave.
template <int ROWS, class Fn>
__device__ inline void each_adapter(int which0, int which1, Fn &&f)
{
    uint64_t left0 = __ballot(which0 >= 0), left1 = ROWS > kWave ? __ballot(which1 >= 0) : 0;
    while (left0 | left1) {
        const int a = left0 ? __builtin_amdgcn_readlane(which0, (int)__builtin_ctzll(left0))
                            : __builtin_amdgcn_readlane(which1, (int)__builtin_ctzll(left1));
        const uint64_t m0 = __ballot(which0 == a), m1 = ROWS > kWave ? __ballot(which1 == a) : 0;
        f(a, m0, m1);
        left0 &= ~m0;
        left1 &= ~m1;
    }
}

__device__ inline int adapter_of(const AdapterArgs &g, int64_t t, bool there)
{
    const int a = there ? g.adapter[t] : -1;
    return a >= 0 && a < g.n ? a : -1;
}

// One wave: U of 16 rows over split_k of K.  RN: rank rounded up.
template <class E, int RN, bool DMA>
__global__ __launch_bounds__(kWave) void down_kernel(AdapterArgs g)
{
    using Ti = Tile<E, true, false, 16, RN, 1, 1>;
    using T = typename E::T;
    __shared__ __attribute__((aligned(16))) T lds[2 * (Ti::kLdsA + Ti::kLdsB)];
    const int lane = threadIdx.x;
    const int t0 = blockIdx.x * 16, k0 = blockIdx.y * g.split_k, K = min(g.split_k, g.K - k0);
    const int which = adapter_of(g, t0 + lane, lane < 16 && t0 + lane < g.T);
    each_adapter<16>(which, -1, [&](int a, uint64_t members, uint64_t) {
        Ti tile;
        tile.clear();
        const Along<E, 16, kWave> x((const T *)g.X + t0 * g.ldx + k0, lane, K,
                                    [&](int, int r) { return members >> r & 1 ? r * g.ldx * E::kBytes : -1; });
        const Across<E, RN, kWave> w((const T *)g.A + a * g.stride_a + k0 * g.lda, lane, K, g.lda, 0, g.R);
        __syncthreads();
        sum_panels<E, DMA, 2>(tile, K, x, w, lds, lane, 0, 0);
        tile.each(0, 0, lane, [&](int r, int c, f32x4 v) {
            if (members >> r & 1) {
                float *u = g.partial + ((int64_t)blockIdx.y * g.T + t0 + r) * g.R + c;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < g.R)
                        u[i] = v[i];
            }
        });
    });
}

// A wave per row.
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
            for (int i = 0; i < g.splits; ++i)
                u[q] += g.partial[((int64_t)i * g.T + t) * g.R + r];
        u[q] *= s;
        top = fmaxf(top, fabsf(u[q]));
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
        // the row's largest value to [1, 2); rows without one as they are
        const int up = top > 0.f && top < INFINITY ? max(ilogbf(top), -100) : 0;
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

template <class E, int BM, int BN, int WM, int WN, bool DMA>
__global__ __launch_bounds__(WM *WN *kWave) void adapters_kernel(AdapterArgs g)
{
    using Ti = Tile<E, true, false, BM, BN, WM, WN>;
    using T = typename E::T;
    constexpr int NT = Ti::kThreads;
    __shared__ __attribute__((aligned(16))) T lds[2 * (Ti::kLdsA + Ti::kLdsB)];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int wm = wave / WN, wn = wave % WN;
    const int total = gridDim.x, per = total / g.xcds, rem = total % g.xcds, xcd = blockIdx.x % g.xcds;
    const int t = xcd * per + min(xcd, rem) + blockIdx.x / g.xcds;   // contiguous tiles per die
    const int m0 = t % g.tiles_m * BM, n0 = t / g.tiles_m * BN;

    Ti tile;
    tile.clear();
    {
        const Along<E, BM, NT> x((const T *)g.X + m0 * g.ldx, tid, g.K,
                                 [&](int, int r) { return m0 + r < g.T ? r * g.ldx * E::kBytes : -1; });
        const Across<E, BN, NT> w((const T *)g.W, tid, g.K, g.ldw, n0, g.N);
        sum_panels<E, DMA, 2>(tile, g.K, x, w, lds, tid, wm, wn);
    }
    if (g.R > 0 && g.n > 0) {
        const int which0 = adapter_of(g, m0 + lane, lane < BM && m0 + lane < g.T);
        const int which1 = adapter_of(g, m0 + 64 + lane, 64 + lane < BM && m0 + 64 + lane < g.T);
        each_adapter<BM>(which0, which1, [&](int a, uint64_t members0, uint64_t members1) {
            auto member = [&](int r) { return (r < 64 ? members0 >> r : members1 >> (r - 64)) & 1; };
            const Along<E, BM, NT> u((const T *)g.factor + (int64_t)m0 * g.depth, tid, g.depth,
                                     [&](int, int r) { return member(r) ? (int64_t)r * g.depth * E::kBytes : -1; });
            const UpRows<E, BN, NT> b((const T *)g.B + a * g.stride_b, tid, g.depth, g.ldb, n0, g.N, g.R);
            Ti add;
            add.clear();
            __syncthreads();
            sum_panels<E, DMA, 2>(add, g.depth, u, b, lds, tid, wm, wn);
#pragma unroll
            for (int m = 0; m < Ti::kFm; ++m) {
                const int r = wm * (BM / WM) + Ti::Fa::row_of(m, lane % 16);
                if (!member(r))
                    continue;
                const float f = E::kBytes == 4 ? 1.f : g.unscale[m0 + r];
#pragma unroll
                for (int n = 0; n < Ti::kFn; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tile.acc[m][n][i] = fmaf(f, add.acc[m][n][i], tile.acc[m][n][i]);
            }
        });
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

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Workgroups along K of the down-projection: about a thousand waves in all,
// at least four panels each.
int down_splits(int T, int K, int panel)
{
    const int64_t tiles = ceil_div(T, 16), panels = ceil_div(K, panel);
    int64_t s = 1024 / tiles;
    if (s > panels / 4)
        s = panels / 4;
    return (int)(s < 1 ? 1 : s > 32 ? 32 : s);
}

struct Workspace {
    size_t partial, factor, unscale, bytes;   // offsets
};
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

template <class E>
Workspace workspace(int T, int K, int R)
{
    Workspace w;
    w.partial = 0;
    w.factor = round16((size_t)down_splits(T, K, panel_deep<E>()) * (size_t)T * (size_t)R * 4);
    w.unscale = w.factor + round16((size_t)T * (size_t)factor_depth<E>(R) * E::kBytes);
    w.bytes = w.unscale + round16((size_t)T * 4);
    return w;
}

template <class E, int RN>
void launch_down(const AdapterArgs &g, bool dma, hipStream_t stream)
{
    const dim3 grid((unsigned)ceil_div(g.T, 16), (unsigned)g.splits);
    if (dma)
        down_kernel<E, RN, true><<<grid, kWave, 0, stream>>>(g);
    else
        down_kernel<E, RN, false><<<grid, kWave, 0, stream>>>(g);
}

template <class E, int BM, int BN, int WM, int WN>
int launch_tiles(AdapterArgs g, bool dma, hipStream_t stream)
{
    const int64_t tm = ceil_div(g.T, BM), tn = ceil_div(g.N, BN);
    if (tm * tn > (int64_t)UINT32_MAX / 256)
        return GEMM_F32_ERR_DIM;
    g.tiles_m = (int)tm;
    g.tiles_n = (int)tn;
    if (dma)
        adapters_kernel<E, BM, BN, WM, WN, true><<<(int)(tm * tn), WM * WN * kWave, 0, stream>>>(g);
    else
        adapters_kernel<E, BM, BN, WM, WN, false><<<(int)(tm * tn), WM * WN * kWave, 0, stream>>>(g);
    return launched();
}

// A grid has fewer than 2^32 threads, and there is a wave per token.
constexpr int kMaxTokens = 1 << 25;

// Most rows of an operand that one panel's offsets span (a tile's, or a panel's depth).
constexpr int kPanelRows = 256;

bool short_ld(int64_t ld, int cols) { return ld < at_least_one(cols); }

}  // namespace
}  // namespace rows

using namespace rows;

extern "C" {

size_t gemm_f32_adapters_ws_size(int type, int T, int N, int K, int R)
{
    if (T <= 0 || T > kMaxTokens || N <= 0 || K < 0 || R <= 0 || R > GEMM_F32_MAX_RANK)
        return 0;
    size_t bytes = 0;
    with_type(type, [&](auto e) { bytes = workspace<decltype(e)>(T, K, R).bytes; });
    return bytes;
}

int gemm_f32_adapters(int type, int T, int N, int K, int R, int n, const void *X, int ldx, const void *W, int ldw,
                      const void *A, int lda, int64_t stride_a, const void *B, int ldb, int64_t stride_b,
                      const int *adapter, const float *scale, void *Y, int ldy, void *ws, size_t ws_bytes,
                      hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (T < 0 || T > kMaxTokens || N < 0 || K < 0 || R < 0 || R > GEMM_F32_MAX_RANK || n < 0)
        return GEMM_F32_ERR_DIM;
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
    const size_t need = low ? gemm_f32_adapters_ws_size(type, T, N, K, R) : 0;
    if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned_to(ws, 16)))
        return GEMM_F32_ERR_WORKSPACE;

    const bool dma_x = dma_rows(type, X, ldx, kPanelRows);
    const bool dma_main = dma_x && dma_rows(type, W, ldw, kPanelRows) &&
                          (!low || (dma_rows(type, B, ldb, kPanelRows) && (n == 1 || stride_b * b % 4 == 0)));
    const bool dma_down = dma_x && low && dma_rows(type, A, lda, kPanelRows) && (n == 1 || stride_a * b % 4 == 0);
    int rc = GEMM_F32_OK;
    with_type(type, [&](auto e) {
        using E = decltype(e);
        AdapterArgs g{};
        g.X = X, g.W = W, g.A = A, g.B = B, g.Y = Y;
        g.adapter = adapter, g.scale = scale;
        g.ldx = ldx, g.ldw = ldw, g.lda = lda, g.ldb = ldb, g.ldy = ldy;
        g.stride_a = stride_a, g.stride_b = stride_b;
        g.T = T, g.N = N, g.K = K, g.R = R, g.n = n;
        g.xcds = gemm_f32_internal::current_device().xcds;
        g.vector_y = vector_rows(type, Y, ldy, 0, N);
        if (low) {
            const Workspace w = workspace<E>(T, K, R);
            g.partial = (float *)((char *)ws + w.partial);
            g.factor = (char *)ws + w.factor;
            g.unscale = (float *)((char *)ws + w.unscale);
            g.depth = factor_depth<E>(R);
            g.splits = down_splits(T, K, panel_deep<E>());
            // whole panels, so that every split starts on a 16-byte boundary
            g.split_k = (int)(ceil_div(ceil_div(K, g.splits), panel_deep<E>()) * panel_deep<E>());
            if (g.split_k > 0)
                g.splits = (int)ceil_div(K, g.split_k);
            if (R <= 16)
                launch_down<E, 16>(g, dma_down, stream);
            else if (R <= 32)
                launch_down<E, 32>(g, dma_down, stream);
            else if (R <= 64)
                launch_down<E, 64>(g, dma_down, stream);
            else if (R <= 128)
                launch_down<E, 128>(g, dma_down, stream);
            else
                launch_down<E, 256>(g, dma_down, stream);
            factor_kernel<E><<<(unsigned)ceil_div(T, kFactorThreads / kWave), kFactorThreads, 0, stream>>>(g);
            rc = launched();
            if (rc != GEMM_F32_OK)
                return;
        }
        // Up to 16 rows: tiles of 16, which read W once without spending
        // matrix instructions on rows that are not there.
        rc = T <= 16 ? launch_tiles<E, 16, 128, 1, 4>(g, dma_main, stream) : launch_tiles<E, 128, 128, 2, 2>(g, dma_main, stream);
    });
    return rc;
}

}  // extern "C"
