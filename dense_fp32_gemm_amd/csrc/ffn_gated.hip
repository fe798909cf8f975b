// Gated projections per group of rows, and the gate's gradient
// (include/gemm_f32_ffn.h).
//
//  * gated_kernel: tiles of rows_tile.h whose second operand holds as many columns of the
//    gate as of what it gates, side by side in each wave's part, so that both sums of an
//    output are in one lane and their product is the epilogue.  8192 rows, 2 x 4096 columns, K = 2048, bf16: 218 us, 1260
//    TFLOP/s (torch.mm of that size 213, without the gate), 239 with the sums kept; K = 4096: 400 and 400.  Panels as
//    the plain product's, so bound as that is.  A launch of one workgroup a compute unit that loads the next
//    tile's first panels under the last one's stores was not faster (226 against 227, 246 against 244 at the time).
//  * gate_grad_kernel: element by element, bound by HBM (16384 x 1024 bf16, 168 MB: 25-28 us, 6.0-6.6 TB/s).
//
// pre is rounded to the type where it is kept: the gradient is that of the rounded sums (off by half a step of
// each), and costs half of what binary32 would move.  dpre is rounded once more, as an operand of the
// products that follow, whose matrix instructions take no other (dX and dW: the root of two roundings' squares, 2.3e-3
// against 1.7e-3 in the 2-norm for bf16).

#include "ffn_gate.h"
#include "rows_groups.h"

namespace ffn {
namespace {

struct GatedArgs {
    GroupedArgs g;           // N: columns of H; C: H
    void *pre;               // NULL: not kept
    int64_t ldp;
    bool vector_p;
};

// Columns of a panel: each wave's BN / WN are half the gate's, half the others'.  16-bit types:
// the first blocks of 16 and the rest.  binary32: four and four in turn, as a lane holds eight
// neighbouring ones of the two blocks that are read together (no tile here reads four).
template <class E, int BN, int NT, int WN>
struct AcrossPair : Across<E, BN, NT> {
    using Base = Across<E, BN, NT>;
    static constexpr int kWide = BN / WN, kHalf = kWide / 2;
    static_assert(E::kBytes == 2 ? kHalf % 16 == 0 : kWide % 32 == 0, "a lane holds both of a pair");
    int N;
    __device__ inline AcrossPair(const typename E::T *base, int tid, int K, int64_t ld, int first, int N_)
        : Base(base, tid, K, ld, first, 2 * N_), N(N_)
    {
    }
    __device__ inline int col(int i) const
    {
        const int p = Base::col(i) - this->first, q = p % kWide, part = p / kWide * kHalf + this->first;
        if constexpr (E::kBytes == 2)
            return q < kHalf ? part + q : N + part + q - kHalf;
        else
            return q % 8 < 4 ? part + q / 8 * 4 : N + part + q / 8 * 4;
    }
    __device__ inline int left(int i, int k0) const
    {
        return (Base::kSlots % NT == 0 || this->tid + i * NT < Base::kSlots) && k0 + this->krow(i) < this->K ? 2 * N - col(i) : 0;
    }
    __device__ inline int inside(int i, int k0) const { return left(i, k0); }
    __device__ inline int64_t offset(int i, int) const { return this->krow(i) * this->ld + (int64_t)col(i) * E::kBytes; }
};

// f(row, column of H, 4 neighbouring gates, what they gate) over the lane's results, within the tile.
template <class E, class Ti, class Fn>
__device__ inline void each_pair(const Ti &tile, int wm, int wn, int lane, Fn &&f)
{
    const int i = lane % 16, h = lane / 16, col = wn * (Ti::BN / Ti::WN / 2);
#pragma unroll
    for (int m = 0; m < Ti::kFm; ++m) {
        const int row = wm * (Ti::BM / Ti::WM) + Ti::Fa::row_of(m, i);
        const auto &a = tile.acc[m];
        if constexpr (E::kBytes == 2) {
#pragma unroll
            for (int n = 0; n < Ti::kFn / 2; ++n)
                f(row, col + 16 * n + 4 * h, a[n], a[n + Ti::kFn / 2]);
        } else {
            static_assert(Ti::Fb::kV == 2, "columns of a pair in one lane");
#pragma unroll
            for (int n = 0; n < Ti::kFn; n += 2)
                f(row, col + 8 * n + 4 * h, f32x4{a[n][0], a[n + 1][0], a[n][1], a[n + 1][1]},
                  f32x4{a[n][2], a[n + 1][2], a[n][3], a[n + 1][3]});
        }
    }
}

// act(gate) * what it gates in the gate's place (see each_pair()).
template <class E, int GATE, class Ti>
__device__ inline void gate_pairs(Ti &tile)
{
#pragma unroll
    for (int m = 0; m < Ti::kFm; ++m)
#pragma unroll
        for (int n = 0; n < Ti::kFn; ++n) {
            constexpr int kUp = E::kBytes == 2 ? Ti::kFn / 2 : 0;
            if (E::kBytes == 2 && n >= kUp)
                continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (E::kBytes == 4 && r >= 2)
                    continue;                        // binary32: the others stand two registers on
                const int up = E::kBytes == 2 ? r : r + 2;
                tile.acc[m][n][r] = gate<GATE>(tile.acc[m][n][r]) * tile.acc[m][n + kUp][up];
            }
        }
}

// One tile: places m0 .. m_end - 1, columns n0 .. n0 + BN / 2 of H.
template <class E, int GATE, int BM, int BN, int WM, int WN, int S, bool DMA>
__device__ inline void gated_tile(const GatedArgs &args, int group, int m0, int m_end, int n0, typename E::T *lds)
{
    using Ti = Tile<E, true, false, BM, BN, WM, WN>;
    using T = typename E::T;
    constexpr int NT = Ti::kThreads;
    const GroupedArgs &g = args.g;
    if (m0 >= m_end || n0 >= g.N)
        return;                                      // the whole workgroup
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / WN, wn = wave % WN;
    Ti tile;
    tile.clear();
    using Src = Along<E, BM, NT>;
    int row[Src::kCount];                            // of X; the loads side by side, then the rest
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
    const Src a((const T *)g.A, tid, g.K, g.lda, g.rows,
                [&](int i, int r) { return m0 + r < m_end && row[i] < g.rows ? row[i] * g.lda * E::kBytes : -1; });
    const AcrossPair<E, BN, NT, WN> b((const T *)g.B + group * g.stride, tid, g.K, g.ldb, n0, g.N);
    sum_panels<E, DMA, S>(tile, g.K, a, b, lds, tid, wm, wn);
    auto each = [&](auto &&f) {                      // of the pairs that are inside
        each_pair<E>(tile, wm, wn, lane, [&](int r, int c, f32x4 x, f32x4 u) {
            if (m0 + r < m_end && n0 + c < g.N)
                f((int64_t)(m0 + r), n0 + c, x, u);
        });
    };
    // (wide and narrow stores apart: merged, the compiler makes pieces of the wide ones, which doubled the
    // time of the stores)
    if (args.pre != nullptr) {
        auto write = [&](auto vec) {
            each([&](int64_t m, int n, f32x4 x, f32x4 u) {
                T *p = (T *)args.pre + m * args.ldp + n;
                store4<E, decltype(vec)::value>(p, x, g.N - n);
                store4<E, decltype(vec)::value>(p + g.N, u, g.N - n);
            });
        };
        args.vector_p ? write(std::true_type{}) : write(std::false_type{});
    }
    gate_pairs<E, GATE>(tile);
    auto write = [&](auto vec) {
        each([&](int64_t m, int n, f32x4 y, f32x4) { store4<E, decltype(vec)::value>((T *)g.C + m * g.ldc + n, y, g.N - n); });
    };
    g.vector_c ? write(std::true_type{}) : write(std::false_type{});
}

template <class E, int GATE, int BM, int BN, int WM, int WN, int S, bool CUT, bool DMA>
__global__ __launch_bounds__(WM *WN *kWave, 2) void gated_kernel(GatedArgs args)
{
    constexpr int kPanel = (BM + BN) * kDeep16 * E::kChunk;
    // (S = 2) two panels of the whole tile, three of a half, four of a quarter
    __shared__ __attribute__((aligned(16))) typename E::T lds[CUT && DMA ? 9 * kPanel / 4 : (DMA ? S : 2) * kPanel];
    static_assert(!CUT || (S == 2 && BM == BN), "panels of cut tiles");
    const GroupedArgs &g = args.g;
    // Rising offsets never have more tiles than the grid has; others are cut there.
    const int total = min(row_tiles(g, BM), g.most_m) * g.tiles_n;
    Part part{-1, 1, 0};
    if constexpr (CUT)
        part = part_of(blockIdx.x, total, g.slots, g.xcds);
    else if ((int)blockIdx.x < total)
        part.tile = die_contiguous(blockIdx.x, total, g.xcds);
    if (part.tile < 0)
        return;                                      // the whole workgroup
    const Place p = locate(g, BM, BM == 256, part.tile);
    const int m0 = p.lo + p.tm * BM, n0 = p.tn * (BN / 2);
    if (!CUT || part.cut == 1)
        gated_tile<E, GATE, BM, BN, WM, WN, S, DMA>(args, p.group, m0, p.hi, n0, lds);
    if constexpr (CUT) {
        if (part.cut == 2)
            gated_tile<E, GATE, BM / 2, BN, WM, WN, 3, DMA>(args, p.group, m0 + part.piece * (BM / 2), p.hi, n0, lds);
        else if (part.cut == 4)
            gated_tile<E, GATE, BM / 2, BN / 2, WM, WN, 4, DMA>(args, p.group, m0 + part.piece % 2 * (BM / 2), p.hi,
                                                                   n0 + part.piece / 2 * (BN / 4), lds);
    }
}

// ---------------------------------------------------------------------------
// The gate's gradient
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

struct GateGradArgs {
    const void *pre, *dH;
    void *dpre;
    int64_t ldp, lddh, lddp;
    int P, N;
    int per_row;             // threads of a row: a power of two
};

template <class E, bool VEC, int GATE>
__global__ __launch_bounds__(kGradThreads) void gate_grad_kernel(GateGradArgs g)
{
    using T = typename E::T;
    const int rows = kGradThreads / g.per_row, j = threadIdx.x % g.per_row;
    for (int64_t p = (int64_t)blockIdx.x * rows + threadIdx.x / g.per_row; p < g.P; p += (int64_t)gridDim.x * rows) {
        const T *pre = (const T *)g.pre + p * g.ldp, *dh = (const T *)g.dH + p * g.lddh;
        T *out = (T *)g.dpre + p * g.lddp;
        for (int n = j * E::kChunk; n < g.N; n += g.per_row * E::kChunk) {
            Chunk<E> a, u, d, da, du;
            a.raw = load_chunk<E, VEC>(pre + n, g.N - n);
            u.raw = load_chunk<E, VEC>(pre + g.N + n, g.N - n);
            d.raw = load_chunk<E, VEC>(dh + n, g.N - n);
#pragma unroll
            for (int e = 0; e < E::kChunk; ++e) {
                float value, slope;
                gate_slope<GATE>((float)a.e[e], value, slope);
                da.e[e] = (T)((float)d.e[e] * (float)u.e[e] * slope);
                du.e[e] = (T)((float)d.e[e] * value);
            }
            store_chunk<E, VEC>(out + n, da, g.N - n);
            store_chunk<E, VEC>(out + g.N + n, du, g.N - n);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <class E, int GATE, int BM, int BN, int WM, int WN, int S, int PER_CU>
int launch_tile(GatedArgs a, bool dma, hipStream_t stream, bool go)
{
    GroupedArgs &g = a.g;
    g.tiles_n = (int)ceil_div(g.N, BN / 2);
    // Every group ends in at most one partial tile.
    const int64_t tiles_m = g.P / BM + (g.G < g.P ? g.G : g.P);
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
        gated_kernel<E, GATE, BM, BN, WM, WN, S, kCut, true><<<(int)grid, WM * WN * kWave, 0, stream>>>(a);
    else
        gated_kernel<E, GATE, BM, BN, WM, WN, S, kCut, false><<<(int)grid, WM * WN * kWave, 0, stream>>>(a);
    return launched();
}

// Tiles as for the plain product of 2N columns (see launch_grouped()), but the 16-bit types take 256 x 256
// tiles, which are cut, as soon as there are more 64 x 128 ones than compute units and they do not pad most groups by
// half (us for 64 x 128 and 256 x 256 tiles: one group, 2 x 4096 columns, K = 2048: 256 rows 17.9 and
// 21.4, 512 rows 27.4 and 23.9, 2048 rows 85 and 57; 2 x 1024 columns: 1024 rows 17.4 and 20.6, 1536 rows 25.2 and 21.2;
// 16 groups: 2048 rows 30.6 and 32.4, 4096 rows 48.6 and 37.2).
template <int GATE>
int launch_gated(int type, const GatedArgs &a, bool dma, hipStream_t stream, bool go)
{
    int rc = GEMM_F32_OK;
    const GroupedArgs &g = a.g;
    with_type(type, [&](auto e) {
        using E = decltype(e);
        if (g.P <= (E::kBytes == 4 ? 64 : 32) * (int64_t)g.G) {
            rc = launch_tile<E, GATE, 32, 64, 2, 2, 4, 0>(a, dma, stream, go);
        } else if constexpr (E::kBytes == 4) {
            rc = launch_tile<E, GATE, 64, 64, 2, 2, 2, 0>(a, dma, stream, go);
        } else {
            if (g.P > 128 * (int64_t)g.G && ceil_div(g.P, 64) * ceil_div(g.N, 64) > gemm_f32_internal::current_device().cus)
                rc = launch_tile<E, GATE, 256, 256, 2, 4, 2, 1>(a, dma, stream, go);
            else
                rc = launch_tile<E, GATE, 64, 128, 2, 2, 3, 0>(a, dma, stream, go);
        }
    });
    return rc;
}

int launch_gated(int type, int gate, const GatedArgs &a, bool dma, hipStream_t stream, bool go = true)
{
    switch (gate) {
    case GEMM_F32_GATE_GELU: return launch_gated<GEMM_F32_GATE_GELU>(type, a, dma, stream, go);
    case GEMM_F32_GATE_GELU_TANH: return launch_gated<GEMM_F32_GATE_GELU_TANH>(type, a, dma, stream, go);
    default: return launch_gated<GEMM_F32_GATE_SILU>(type, a, dma, stream, go);
    }
}

bool bad_pair(int N) { return N < 0 || N > kMaxSize / 2; }

}  // namespace
}  // namespace ffn

using namespace ffn;

extern "C" {

int gemm_f32_gated(int type, int gate, int G, int P, int N, int K, const int *offsets, const int *order, int per_row, int rows,
                   const void *X, int ldx, const void *W, int ldw, int64_t stride_w, void *H, int ldh, void *pre, int ldp,
                   hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (G < 0 || bad_size(P) || bad_pair(N) || bad_size(K) || rows < 0 || (order == nullptr && rows < P))
        return GEMM_F32_ERR_DIM;
    GatedArgs a{{offsets, order, X, W, H, ldx, ldw, ldh, stride_w, G, P, rows, Divisor(1), 0, N, K,
                 gemm_f32_internal::current_device().xcds, vector_rows(type, H, ldh, 0, N), 0, 0, 0},
                pre, ldp, vector_rows(type, pre, ldp, 0, N)};
    const int rc = launch_gated(type, gate, a, false, nullptr, false);
    if (rc != GEMM_F32_OK)
        return rc;
    if (short_ld(ldx, K) || short_ld(ldw, 2 * N) || short_ld(ldh, N) || (pre != nullptr && short_ld(ldp, 2 * N)) ||
        short_stride(stride_w, G, K, ldw))
        return GEMM_F32_ERR_LD;
    if (!known_gate(gate) || (order != nullptr && per_row < 1))
        return GEMM_F32_ERR_OPTION;
    if (G == 0 || P == 0 || N == 0)
        return GEMM_F32_OK;
    if (no_offsets(offsets, G) || H == nullptr || (K > 0 && ((X == nullptr && rows > 0) || W == nullptr)))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(offsets, 4) || !aligned_to(order, 4) || !aligned_to(X, b) || !aligned_to(W, b) || !aligned_to(H, b) ||
        !aligned_to(pre, b))
        return GEMM_F32_ERR_ALIGN;
    if (order != nullptr)
        a.g.per_row = Divisor(per_row);
    // the second half of W's columns has to start on four bytes too
    const bool dma = dma_rows(type, X, ldx, rows) && dma_rows(type, W, ldw, kPanelRows) && stride_w * b % 4 == 0 && N * (int64_t)b % 4 == 0;
    return launch_gated(type, gate, a, dma, stream);
}

int gemm_f32_gate_grad(int type, int gate, int P, int N, const void *pre, int ldp, const void *dH, int lddh, void *dpre,
                       int lddp, hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (bad_size(P) || bad_pair(N))
        return GEMM_F32_ERR_DIM;
    if (short_ld(ldp, 2 * N) || short_ld(lddh, N) || short_ld(lddp, 2 * N))
        return GEMM_F32_ERR_LD;
    if (!known_gate(gate))
        return GEMM_F32_ERR_OPTION;
    if (P == 0 || N == 0)
        return GEMM_F32_OK;
    if (pre == nullptr || dH == nullptr || dpre == nullptr)
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(pre, b) || !aligned_to(dH, b) || !aligned_to(dpre, b))
        return GEMM_F32_ERR_ALIGN;
    const bool vec = chunk_rows(type, pre, ldp, N) && chunk_rows(type, dH, lddh, N) && chunk_rows(type, dpre, lddp, N);
    with_type(type, [&](auto e) {
        using E = decltype(e);
        int per_row = 1;
        while (per_row < kGradThreads && per_row * E::kChunk < N)
            per_row *= 2;
        const GateGradArgs g{pre, dH, dpre, ldp, lddh, lddp, P, N, per_row};
        const int64_t need = ceil_div(P, kGradThreads / per_row);
        const int grid = (int)(need < kMaxTiles ? need : kMaxTiles);
        auto launch = [&](auto v, auto kind) {
            gate_grad_kernel<E, decltype(v)::value, decltype(kind)::value><<<grid, kGradThreads, 0, stream>>>(g);
        };
        auto pick = [&](auto kind) { vec ? launch(std::true_type{}, kind) : launch(std::false_type{}, kind); };
        if (gate == GEMM_F32_GATE_GELU)
            pick(Gate<GEMM_F32_GATE_GELU>{});
        else if (gate == GEMM_F32_GATE_GELU_TANH)
            pick(Gate<GEMM_F32_GATE_GELU_TANH>{});
        else
            pick(Gate<GEMM_F32_GATE_SILU>{});
    });
    return launched();
}

}  // extern "C"
