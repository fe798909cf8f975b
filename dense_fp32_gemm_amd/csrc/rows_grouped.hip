// Products per group of rows, their gradients, and the weighted sum of a
// token's results (include/gemm_f32_rows.h).
//
//  * grouped_kernel<E, OP, ...>: one workgroup per output tile.  Which group a
//    workgroup's tile belongs to is found on the device, from the offsets.
//  * combine_kernel, combine_grad_kernel: one workgroup per token.

#include "rows_groups.h"

namespace rows {
namespace {

enum Op { kForward, kGradX, kGradW };

// Tile t of dW.  A group's tiles cost its number of places, so each die's range of t has a
// slice of every group (both gradients, 4096 x 4 slots over 16 experts of unlike
// shares, 2048 x 2048, bf16: 351 us against 402 with whole groups to a die; 8192 x 2 over 8:
// 343 against 445; 1025 x 2 over 8, 1000 x 1023, binary32: 104 against 136).
__device__ inline Place spread(const GroupedArgs &g, int tiles_m, int t)
{
    const int per = tiles_m * g.tiles_n;
    int s = 0, from = 0, to = per / g.xcds;          // slice s: a group's tiles from .. to - 1
    while (t >= (int64_t)g.G * to) {                 // to reaches per, and t < G * per
        ++s;
        from = to;
        to = (int)((int64_t)per * (s + 1) / g.xcds);
    }
    const int rest = t - g.G * from, r = from + rest % (to - from);
    // two columns of tiles side by side, so that a slice shares rows and columns (the first two
    // cases above: 345 against 351 with one column after the other, 335 against 343)
    const int band = r / (2 * tiles_m), q = r - band * 2 * tiles_m, wide = min(2, g.tiles_n - 2 * band);
    return Place{rest / (to - from), 0, 0, q / wide, 2 * band + q % wide};
}

// One tile: rows m0 .. m_end - 1 (places; of dW: rows of the matrix), columns from n0 on.
template <class E, Op OP, int BM, int BN, int WM, int WN, int S, bool DMA>
__device__ inline void grouped_tile(const GroupedArgs &g, int group, int lo, int hi, int m0, int m_end, int n0,
                                    typename E::T *lds, uint32_t *ahead)
{
    constexpr bool kAlongA = OP != kGradW, kAlongB = OP == kGradX;
    using Ti = Tile<E, kAlongA, kAlongB, BM, BN, WM, WN>;
    using T = typename E::T;
    constexpr int NT = Ti::kThreads;
    if (m0 >= m_end || n0 >= g.N)
        return;                                      // the whole workgroup
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / WN, wn = wave % WN;
    const T *A = (const T *)g.A, *B = (const T *)g.B;

    Ti tile;
    tile.clear();
    if constexpr (OP == kForward) {
        using Src = Along<E, BM, NT>;
        int row[Src::kCount];                        // of X; the loads side by side, then the rest
        if (g.order != nullptr) {
#pragma unroll
            for (int i = 0; i < Src::kCount; ++i)
                row[i] = g.order[min(m0 + Src::row_of(i, tid), m_end - 1)];
#pragma unroll
            for (int i = 0; i < Src::kCount; ++i)
                row[i] = row[i] < 0 ? INT32_MAX : g.per_row.of(row[i]);
        } else {
#pragma unroll
            for (int i = 0; i < Src::kCount; ++i)
                row[i] = m0 + Src::row_of(i, tid);
        }
        const Src a(A, tid, g.K, g.lda, g.rows,
                    [&](int i, int r) { return m0 + r < m_end && row[i] < g.rows ? row[i] * g.lda * E::kBytes : -1; });
        const Across<E, BN, NT> b(B + group * g.stride, tid, g.K, g.ldb, n0, g.N);
        sum_panels<E, DMA, S>(tile, g.K, a, b, lds, tid, wm, wn);
    } else if constexpr (OP == kGradX) {
        const Along<E, BM, NT> a(A + m0 * g.lda, tid, g.K, g.lda, g.P - m0,
                                 [&](int, int r) { return m0 + r < m_end ? r * g.lda * E::kBytes : -1; });
        const Along<E, BN, NT> b(B + group * g.stride + n0 * g.ldb, tid, g.K, g.ldb, g.N - n0,
                                 [&](int, int r) { return n0 + r < g.N ? r * g.ldb * E::kBytes : -1; });
        sum_panels<E, DMA, S>(tile, g.K, a, b, lds, tid, wm, wn);
    } else {
        const int *list = g.order != nullptr ? g.order + lo : nullptr;
        const T *X = g.order != nullptr ? A : A + lo * g.lda;
        const int rows = g.order != nullptr ? g.rows : hi - lo;
        const Gathered<E, BM, NT> a(X, tid, hi - lo, g.lda, m0, g.M, list, g.per_row, rows, ahead);
        const Across<E, BN, NT> b(B + lo * g.ldb, tid, hi - lo, g.ldb, n0, g.N);
        sum_panels<E, DMA, S>(tile, hi - lo, a, b, lds, tid, wm, wn);
    }

    T *C = (T *)g.C + (OP == kGradW ? group * g.stride : 0);
    auto store = [&](auto vec) {
        tile.each(wm, wn, lane, [&](int r, int c, f32x4 v) {
            const int m = m0 + r, n = n0 + c;
            if (m < m_end && n < g.N)
                store4<E, decltype(vec)::value>(C + (int64_t)m * g.ldc + n, v, g.N - n);
        });
    };
    if (g.vector_c)
        store(std::true_type{});
    else
        store(std::false_type{});
}

template <class E, Op OP, int BM, int BN, int WM, int WN, int S, bool CUT, bool DMA>
__global__ __launch_bounds__(WM *WN *kWave, 2) void grouped_kernel(GroupedArgs g)
{
    constexpr int kPanel = (BM + BN) * kDeep16 * E::kChunk;
    // (S = 2) two panels of the whole tile, three of a half, four of a quarter
    __shared__ __attribute__((aligned(16))) typename E::T lds[CUT && DMA ? 9 * kPanel / 4 : (DMA ? S : 2) * kPanel];
    static_assert(!CUT || (S == 2 && BM == BN), "panels of cut tiles");
    __shared__ uint32_t ahead[OP == kGradW && DMA ? 1024 : 1];
    const int tiles_m = OP == kGradW ? (g.M + BM - 1) / BM : 0;
    // Rising offsets never have more tiles than the grid has; others are cut there.
    const int total = OP == kGradW ? g.G * tiles_m * g.tiles_n : min(row_tiles(g, BM), g.most_m) * g.tiles_n;
    Part part{-1, 1, 0};
    if constexpr (CUT)
        part = part_of(blockIdx.x, total, g.slots, g.xcds);
    else if ((int)blockIdx.x < total)
        part.tile = die_contiguous(blockIdx.x, total, g.xcds);
    if (part.tile < 0)
        return;                                      // the whole workgroup
    Place p;
    if constexpr (OP == kGradW) {
        const Place q = spread(g, tiles_m, part.tile);
        p.group = q.group, p.tm = q.tm, p.tn = q.tn;
        group_range(g.offsets, p.group, g.P, p.lo, p.hi);
        p.lo = __builtin_amdgcn_readfirstlane(p.lo);
        p.hi = __builtin_amdgcn_readfirstlane(p.hi);
    } else {
        p = locate(g, BM, BM == 256 && (OP == kForward || g.G == 1), part.tile);
    }
    const int m0 = (OP == kGradW ? 0 : p.lo) + p.tm * BM, m_end = OP == kGradW ? g.M : p.hi, n0 = p.tn * BN;
    if (!CUT || part.cut == 1)
        grouped_tile<E, OP, BM, BN, WM, WN, S, DMA>(g, p.group, p.lo, p.hi, m0, m_end, n0, lds, ahead);
    if constexpr (CUT) {
        if (part.cut == 2)
            grouped_tile<E, OP, BM / 2, BN, WM, WN, 3, DMA>(g, p.group, p.lo, p.hi, m0 + part.piece * (BM / 2), m_end,
                                                               n0, lds, ahead);
        else if (part.cut == 4)
            grouped_tile<E, OP, BM / 2, BN / 2, WM, WN, 4, DMA>(g, p.group, p.lo, p.hi,
                                                                   m0 + part.piece % 2 * (BM / 2), m_end,
                                                                   n0 + part.piece / 2 * (BN / 2), lds, ahead);
    }
}

// ---------------------------------------------------------------------------
// Weighted sum of a token's results
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;

struct CombineArgs {
    const int *position;
    const float *weight;
    const void *Y;
    const void *dout;
    void *out;
    void *dY;
    float *dweight;
    int64_t ldy, ldo, lddo, lddy;
    int T, k, N, P;
};

// kSlots results' loads in flight a thread; the sum stays in the order of j.  Bound by HBM
// reads in rows' order of arrival: 8192 tokens, k = 8, N = 2048, bf16: 70-76 us for 302 MB,
// 4.1 TB/s.
template <class E, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineArgs g)
{
    using T = typename E::T;
    constexpr int kSlots = 8;
    for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
        const int *position = g.position + t * g.k;
        for (int n = threadIdx.x * E::kChunk; n < g.N; n += kCombineThreads * E::kChunk) {
            float sum[E::kChunk] = {};
            for (int j0 = 0; j0 < g.k; j0 += kSlots) {
                Chunk<E> y[kSlots];
                float w[kSlots];
                bool there[kSlots];
#pragma unroll
                for (int q = 0; q < kSlots; ++q) {
                    const int p = j0 + q < g.k ? position[j0 + q] : -1;
                    there[q] = p >= 0 && p < g.P;
                    w[q] = there[q] && g.weight != nullptr ? g.weight[t * g.k + j0 + q] : 1.f;
                    y[q].raw = load_chunk<E, VEC>((const T *)g.Y + (there[q] ? p : 0) * g.ldy + n, there[q] ? g.N - n : 0);
                }
#pragma unroll
                for (int q = 0; q < kSlots; ++q)
                    if (there[q]) {
#pragma unroll
                        for (int i = 0; i < E::kChunk; ++i)
                            sum[i] = fmaf(w[q], (float)y[q].e[i], sum[i]);
                    }
            }
            Chunk<E> o;
#pragma unroll
            for (int i = 0; i < E::kChunk; ++i)
                o.e[i] = (T)sum[i];
            store_chunk<E, VEC>((T *)g.out + t * g.ldo + n, o, g.N - n);
        }
    }
}

// Bound by HBM: the same sizes 108-111 us for 570 MB, 5.2 TB/s.
// The inner product in binary32: a thread's chunks, then the waves' lanes, then the waves.
template <class E, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void combine_grad_kernel(CombineArgs g)
{
    using T = typename E::T;
    __shared__ float part[kCombineThreads / kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
        for (int j = 0; j < g.k; ++j) {
            const int p = g.position[t * g.k + j];
            const bool there = p >= 0 && p < g.P;
            const float w = g.weight != nullptr ? g.weight[t * g.k + j] : 1.f;
            float sum = 0.f;
            if (there) {
                for (int n = threadIdx.x * E::kChunk; n < g.N; n += kCombineThreads * E::kChunk) {
                    Chunk<E> d;
                    d.raw = load_chunk<E, VEC>((const T *)g.dout + t * g.lddo + n, g.N - n);
                    if (g.dweight != nullptr) {
                        Chunk<E> y;
                        y.raw = load_chunk<E, VEC>((const T *)g.Y + p * g.ldy + n, g.N - n);
#pragma unroll
                        for (int i = 0; i < E::kChunk; ++i)
                            sum = fmaf((float)y.e[i], (float)d.e[i], sum);
                    }
                    if (g.dY != nullptr) {
                        Chunk<E> o;
#pragma unroll
                        for (int i = 0; i < E::kChunk; ++i)
                            o.e[i] = (T)(w * (float)d.e[i]);
                        store_chunk<E, VEC>((T *)g.dY + p * g.lddy + n, o, g.N - n);
                    }
                }
            }
            if (g.dweight == nullptr)
                continue;
#pragma unroll
            for (int d = kWave / 2; d > 0; d /= 2)
                sum += __shfl_xor(sum, d);
            if (lane == 0)
                part[wave] = sum;
            __syncthreads();
            if (threadIdx.x == 0)
                g.dweight[t * g.k + j] = (part[0] + part[1]) + (part[2] + part[3]);
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static_assert(kCombineThreads <= 512, "grid limit");
int token_grid(int T) { return T < kMaxTiles ? T : (int)kMaxTiles; }

// PER_CU: workgroups of a kernel that cuts its last tiles on a compute unit (0: it does not).
// Without `go` it says whether the tiles fit a grid.
template <class E, Op OP, int BM, int BN, int WM, int WN, int S, int PER_CU>
int launch_tile(GroupedArgs g, bool dma, hipStream_t stream, bool go)
{
    g.tiles_n = (int)ceil_div(g.N, BN);
    // Every group ends in at most one partial tile.
    const int64_t tiles_m = OP == kGradW ? g.G * ceil_div(g.M, BM) : g.P / BM + (g.G < g.P ? g.G : g.P);
    g.slots = (int)gemm_f32_internal::current_device().cus * PER_CU;
    // Cutting the last round adds at most three pieces for a quarter of the slots.
    const int64_t grid = (tiles_m < kMaxTiles ? tiles_m : kMaxTiles) * g.tiles_n + g.slots;
    if (tiles_m > kMaxTiles || grid > kMaxTiles)
        return GEMM_F32_ERR_DIM;
    if (!go || tiles_m * g.tiles_n == 0)
        return GEMM_F32_OK;
    g.most_m = (int)tiles_m;
    constexpr bool kCut = PER_CU > 0;
    if (dma)
        grouped_kernel<E, OP, BM, BN, WM, WN, S, kCut, true><<<(int)grid, WM * WN * kWave, 0, stream>>>(g);
    else
        grouped_kernel<E, OP, BM, BN, WM, WN, S, kCut, false><<<(int)grid, WM * WN * kWave, 0, stream>>>(g);
    return launched();
}

// Tiles by the rows a group has on average and by how many tiles there are (us a
// call, one MI355X, K = 2048 -> N = 1024 unless said):
//  * up to 32 rows a group (binary32: 64), a tile of 32 x 64: many workgroups, each weight
//    read once or twice (32 rows over 32 groups, bf16: 13.4 against 17.2 for 64 x 128; 512 rows
//    over 16 groups: 17.7 against 17.8, 768 rows: 19.7 against 18.0; binary32, 1024
//    rows over 16 groups: 60 against 69 for 64 x 64, 1536 rows: equal);
//  * binary32 else: 64 x 64 (4096 rows over 8 groups, N = 2048: 282; with slower loads 293 against 310 for 128 x 64
//    and 312 for 128 x 128, whose last round leaves more units idle);
//  * 16-bit types, 256 x 256 tiles for three fifths of the compute units or
//    more: those, the last round cut (2000 rows over 8 groups, N = 4096: 56 against 76
//    for 64 x 128; 65536 rows over 64: 288 against 355 for 128 x 128). A compute unit
//    was seen to take up to about 16 bytes a clock of panels from L2; the largest tile needs
//    the fewest per product, 12 to 14 at its rate here (961 TFLOP/s, an eighth of the rows padding);
//  * fewer: 64 x 128 (4096 rows over 8 groups, K = N = 1024: 19.4 against 21.6).
template <Op OP>
int launch_grouped(int type, const GroupedArgs &g, bool dma, hipStream_t stream, bool go = true)
{
    int rc = GEMM_F32_OK;
    with_type(type, [&](auto e) {
        using E = decltype(e);
        if constexpr (OP != kGradW) {
            if (g.P <= (E::kBytes == 4 ? 64 : 32) * (int64_t)g.G) {
                rc = launch_tile<E, OP, 32, 64, 1, 4, 4, 0>(g, dma, stream, go);
                return;
            }
        }
        if constexpr (E::kBytes == 4) {
            rc = launch_tile<E, OP, 64, 64, 2, 2, 2, 0>(g, dma, stream, go);
        } else {
            // Half a tile a group is lost on average.
            const int64_t rows = OP == kGradW ? 2 * g.G * ceil_div(g.M, 256) : 2 * (g.P / 256) + (g.G < g.P ? g.G : g.P);
            if ((rows < kMaxTiles ? rows : kMaxTiles) * ceil_div(g.N, 256) * 5 >= 6 * gemm_f32_internal::current_device().cus)
                rc = launch_tile<E, OP, 256, 256, 2, 4, 2, 1>(g, dma, stream, go);
            else
                rc = launch_tile<E, OP, 64, 128, 2, 2, 3, 0>(g, dma, stream, go);
        }
    });
    return rc;
}

// Type and sizes, the number of tiles among them (see launch_tile()).
template <Op OP>
int check_grouped(int type, int G, int P, int N, int K)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (G < 0 || bad_size(P) || bad_size(N) || bad_size(K))
        return GEMM_F32_ERR_DIM;
    const int cols = OP == kGradX ? K : N;
    const GroupedArgs g{nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, 0, 0, G, P, 0, Divisor(1), K, cols, 0, 1, false, 0, 0, 0};
    return launch_grouped<OP>(type, g, false, nullptr, false);
}


}  // namespace
}  // namespace rows

using namespace rows;

extern "C" {

int gemm_f32_grouped(int type, int G, int P, int N, int K, const int *offsets, const int *order, int per_row, int rows,
                     const void *X, int ldx, const void *W, int ldw, int64_t stride_w, void *Y, int ldy,
                     hipStream_t stream)
{
    const int rc = check_grouped<kForward>(type, G, P, N, K);
    if (rc != GEMM_F32_OK)
        return rc;
    if (rows < 0 || (order == nullptr && rows < P))
        return GEMM_F32_ERR_DIM;
    if (short_ld(ldx, K) || short_ld(ldw, N) || short_ld(ldy, N) || short_stride(stride_w, G, K, ldw))
        return GEMM_F32_ERR_LD;
    if (order != nullptr && per_row < 1)
        return GEMM_F32_ERR_OPTION;
    if (G == 0 || P == 0 || N == 0)
        return GEMM_F32_OK;
    if (no_offsets(offsets, G) || Y == nullptr || (K > 0 && ((X == nullptr && rows > 0) || W == nullptr)))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(offsets, 4) || !aligned_to(order, 4) || !aligned_to(X, b) || !aligned_to(W, b) || !aligned_to(Y, b))
        return GEMM_F32_ERR_ALIGN;
    const bool dma = dma_rows(type, X, ldx, rows) && dma_rows(type, W, ldw, kPanelRows) && stride_w * b % 4 == 0;
    const GroupedArgs g{offsets, order, X, W, Y, ldx, ldw, ldy, stride_w, G, P, rows, Divisor(order != nullptr ? per_row : 1), 0, N, K,
                        gemm_f32_internal::current_device().xcds, vector_rows(type, Y, ldy, 0, N), 0, 0, 0};
    return launch_grouped<kForward>(type, g, dma, stream);
}

int gemm_f32_grouped_grad_x(int type, int G, int P, int N, int K, const int *offsets, const void *dY, int lddy,
                            const void *W, int ldw, int64_t stride_w, void *dX, int lddx, hipStream_t stream)
{
    const int rc = check_grouped<kGradX>(type, G, P, N, K);
    if (rc != GEMM_F32_OK)
        return rc;
    if (short_ld(lddy, N) || short_ld(ldw, N) || short_ld(lddx, K) || short_stride(stride_w, G, K, ldw))
        return GEMM_F32_ERR_LD;
    if (G == 0 || P == 0 || K == 0)
        return GEMM_F32_OK;
    if (no_offsets(offsets, G) || dX == nullptr || (N > 0 && (dY == nullptr || W == nullptr)))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(offsets, 4) || !aligned_to(dY, b) || !aligned_to(W, b) || !aligned_to(dX, b))
        return GEMM_F32_ERR_ALIGN;
    const bool dma = dma_rows(type, dY, lddy, kPanelRows) && dma_rows(type, W, ldw, kPanelRows) && stride_w * b % 4 == 0;
    const GroupedArgs g{offsets, nullptr, dY, W, dX, lddy, ldw, lddx, stride_w, G, P, P, Divisor(1), 0, K, N,
                        gemm_f32_internal::current_device().xcds, vector_rows(type, dX, lddx, 0, K), 0, 0, 0};
    return launch_grouped<kGradX>(type, g, dma, stream);
}

int gemm_f32_grouped_grad_w(int type, int G, int P, int N, int K, const int *offsets, const int *order, int per_row,
                            int rows, const void *X, int ldx, const void *dY, int lddy, void *dW, int lddw,
                            int64_t stride_dw, hipStream_t stream)
{
    const int rc = check_grouped<kGradW>(type, G, P, N, K);
    if (rc != GEMM_F32_OK)
        return rc;
    if (rows < 0 || (order == nullptr && rows < P))
        return GEMM_F32_ERR_DIM;
    if (short_ld(ldx, K) || short_ld(lddy, N) || short_ld(lddw, N) || short_stride(stride_dw, G, K, lddw))
        return GEMM_F32_ERR_LD;
    if (order != nullptr && per_row < 1)
        return GEMM_F32_ERR_OPTION;
    if (G == 0 || K == 0 || N == 0)
        return GEMM_F32_OK;
    if (no_offsets(offsets, G) || dW == nullptr || (P > 0 && ((X == nullptr && rows > 0) || dY == nullptr)))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(offsets, 4) || !aligned_to(order, 4) || !aligned_to(X, b) || !aligned_to(dY, b) || !aligned_to(dW, b))
        return GEMM_F32_ERR_ALIGN;
    const bool dma = dma_rows(type, X, ldx, rows) && dma_rows(type, dY, lddy, kPanelRows);
    const GroupedArgs g{offsets, order, X, dY, dW, ldx, lddy, lddw, stride_dw, G, P, rows, Divisor(order != nullptr ? per_row : 1), K, N, 0,
                        gemm_f32_internal::current_device().xcds, vector_rows(type, dW, lddw, stride_dw, N), 0, 0, 0};
    return launch_grouped<kGradW>(type, g, dma, stream);
}

int gemm_f32_combine(int type, int T, int k, int N, int P, const int *position, const float *weight, const void *Y,
                     int ldy, void *out, int ldo, hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (T < 0 || bad_size(k) || bad_size(N) || P < 0)
        return GEMM_F32_ERR_DIM;
    if (short_ld(ldy, N) || short_ld(ldo, N))
        return GEMM_F32_ERR_LD;
    if (T == 0 || N == 0)
        return GEMM_F32_OK;
    if (out == nullptr || (k > 0 && (position == nullptr || (P > 0 && Y == nullptr))))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(position, 4) || !aligned_to(weight, 4) || !aligned_to(Y, b) || !aligned_to(out, b))
        return GEMM_F32_ERR_ALIGN;
    const CombineArgs g{position, weight, Y, nullptr, out, nullptr, nullptr, ldy, ldo, 0, 0, T, k, N, P};
    const bool vec = chunk_rows(type, Y, ldy, N) && chunk_rows(type, out, ldo, N);
    with_type(type, [&](auto e) {
        using E = decltype(e);
        if (vec)
            combine_kernel<E, true><<<token_grid(T), kCombineThreads, 0, stream>>>(g);
        else
            combine_kernel<E, false><<<token_grid(T), kCombineThreads, 0, stream>>>(g);
    });
    return launched();
}

int gemm_f32_combine_grad(int type, int T, int k, int N, int P, const int *position, const float *weight,
                          const void *Y, int ldy, const void *dout, int lddo, void *dY, int lddy, float *dweight,
                          hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (T < 0 || bad_size(k) || bad_size(N) || P < 0)
        return GEMM_F32_ERR_DIM;
    if ((dweight != nullptr && short_ld(ldy, N)) || short_ld(lddo, N) || (dY != nullptr && short_ld(lddy, N)))
        return GEMM_F32_ERR_LD;
    if (T == 0 || k == 0 || (dY == nullptr && dweight == nullptr))
        return GEMM_F32_OK;
    if (position == nullptr || (N > 0 && (dout == nullptr || (dweight != nullptr && P > 0 && Y == nullptr))))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(position, 4) || !aligned_to(weight, 4) || !aligned_to(Y, b) || !aligned_to(dout, b) ||
        !aligned_to(dY, b) || !aligned_to(dweight, 4))
        return GEMM_F32_ERR_ALIGN;
    const CombineArgs g{position, weight, Y, dout, nullptr, dY, dweight, ldy, 0, lddo, lddy, T, k, N, P};
    const bool vec = (dweight == nullptr || chunk_rows(type, Y, ldy, N)) && chunk_rows(type, dout, lddo, N) &&
                     (dY == nullptr || chunk_rows(type, dY, lddy, N));
    with_type(type, [&](auto e) {
        using E = decltype(e);
        if (vec)
            combine_grad_kernel<E, true><<<token_grid(T), kCombineThreads, 0, stream>>>(g);
        else
            combine_grad_kernel<E, false><<<token_grid(T), kCombineThreads, 0, stream>>>(g);
    });
    return launched();
}

}  // extern "C"
