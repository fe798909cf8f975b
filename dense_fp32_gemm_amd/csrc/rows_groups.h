// Products per group of rows: their arguments, and where a group's tiles are.
#ifndef GEMM_F32_ROWS_GROUPS_H
#define GEMM_F32_ROWS_GROUPS_H

#include "rows_tile.h"

namespace rows {

struct GroupedArgs {
    const int *offsets;      // NULL: one group of all places
    const int *order;        // forward, grad_w: rows of A; NULL: the place itself
    const void *A;           // X (forward, grad_w), dY (grad_x)
    const void *B;           // W (forward, grad_x), dY (grad_w)
    void *C;                 // Y, dX, dW
    int64_t lda, ldb, ldc;
    int64_t stride;          // of W (of dW for grad_w)
    int G, P, rows;          // rows: of X
    Divisor per_row;
    int M, N, K;             // grad_w: M x N of dW; else columns N of C, summed K
    int xcds;
    bool vector_c;           // C's rows take stores of four elements
    int tiles_n;
    int most_m;              // row tiles there can be
    int slots;               // workgroups the device holds at once
};

// Group g's range of places, clamped to 0..P; without offsets all of them.
__device__ inline void group_range(const int *offsets, int g, int P, int &lo, int &hi)
{
    if (offsets == nullptr) {
        lo = 0, hi = P;
        return;
    }
    lo = min(max(offsets[g], 0), P);
    hi = min(max(offsets[g + 1], lo), P);
}

struct Place {
    int group, lo, hi;       // the group's places
    int tm, tn;              // row tile within the group, column tile
};

// Row tiles of all groups (64 groups at a time, a lane each), the same in every lane.
__device__ inline int row_tiles(const GroupedArgs &g, int bm)
{
    if (g.offsets == nullptr)
        return (g.P + bm - 1) / bm;
    const int lane = threadIdx.x % kWave;
    int total = 0;
    for (int g0 = 0; g0 < g.G; g0 += kWave) {
        int a = 0, b = 0;
        if (g0 + lane < g.G)
            group_range(g.offsets, g0 + lane, g.P, a, b);
        int n = (b - a + bm - 1) / bm;
#pragma unroll
        for (int d = kWave / 2; d > 0; d /= 2)
            n += __shfl_xor(n, d);
        total += n;
    }
    return __builtin_amdgcn_readfirstlane(total);
}

// Row tiles of a band of 256 x 256 tiles: a die's 32 tiles that run side by side are then 4 x 8 and share rows and
// columns in its L2 (bf16, 8192 rows, 8192 columns, K = 2048: 232 us; bands of 8: 233, whole columns: 242; the gradient
// of X 195 and 204; 32768 rows over 8 groups, 2048 x 2048: 262 and 272).  Whole columns, one after the other, are as
// good or better up to two bands of rows, in the gradient of X of several groups (32768 over 8: 250 us, banded 260;
// 65536 over 64, 2048 -> 1024: 320 and 335), and with 64 x 128 tiles (1500 rows over 8, 2048 x 2048: 24.7 and 28.2).
constexpr int kBand = 4;

// The r-th tile of a group that has `rows` row tiles.
__device__ inline Place tile_of(const GroupedArgs &g, bool banded, Place p, int r, int rows)
{
    if (!banded || rows <= 2 * kBand) {
        p.tn = r / rows;
        p.tm = r - p.tn * rows;
        return p;
    }
    const int from = r / (kBand * g.tiles_n) * kBand, q = r - from * g.tiles_n, high = min(kBand, rows - from);
    p.tn = high == kBand ? q / kBand : q / high;     // (the usual case without a division)
    p.tm = from + q - p.tn * high;
    return p;
}

// Tile t, counted group by group, band by band within a group if they are banded, and column by column within a
// band.  Every wave of the workgroup computes it for itself.
__device__ inline Place locate(const GroupedArgs &g, int bm, bool banded, int t)
{
    if (g.offsets == nullptr)
        return tile_of(g, banded, Place{0, 0, g.P, 0, 0}, t, (g.P + bm - 1) / bm);
    const int lane = threadIdx.x % kWave;
    int before = 0;                                  // row tiles of the groups before
    Place p{0, 0, 0, 0, 0};
    for (int g0 = 0; g0 < g.G; g0 += kWave) {
        int a = 0, b = 0;
        if (g0 + lane < g.G)
            group_range(g.offsets, g0 + lane, g.P, a, b);
        const int n = (b - a + bm - 1) / bm;
        int scan = n;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int x = __shfl_up(scan, d);
            scan += lane >= d ? x : 0;
        }
        const uint64_t past = __ballot(before + scan > t / g.tiles_n);
        if (past) {
            const int at = (int)__builtin_ctzll(past);
            const int mine = __builtin_amdgcn_readlane(n, at);
            const int first = before + __builtin_amdgcn_readlane(scan, at) - mine;
            p = tile_of(g, banded, Place{g0 + at, __builtin_amdgcn_readlane(a, at), __builtin_amdgcn_readlane(b, at), 0, 0},
                       t - first * g.tiles_n, mine);
            break;
        }
        before += __builtin_amdgcn_readlane(scan, kWave - 1);
    }
    // scalars, whatever the compiler makes of the loop
    return Place{__builtin_amdgcn_readfirstlane(p.group), __builtin_amdgcn_readfirstlane(p.lo),
                 __builtin_amdgcn_readfirstlane(p.hi), __builtin_amdgcn_readfirstlane(p.tm),
                 __builtin_amdgcn_readfirstlane(p.tn)};
}

// Most rows of an operand that one panel's offsets span (BM, BN or a panel's depth).
constexpr int kPanelRows = 256;

// Workgroups of a launch: a grid has fewer than 2^32 threads.
constexpr int64_t kMaxTiles = UINT32_MAX / 512;

// K * ldw elements between groups at least (the last row may end at N).
inline bool short_stride(int64_t stride, int G, int K, int64_t ldw) { return G > 1 && stride < K * ldw; }
// Offsets may be left out where there is one group.
inline bool no_offsets(const int *offsets, int G) { return offsets == nullptr && G != 1; }

}  // namespace rows

#endif
