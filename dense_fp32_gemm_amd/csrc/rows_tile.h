// One output tile of a product on the matrix cores, from panels in LDS.
//
// Panels are kDeep (128 bytes of) elements deep in the summed index.  An operand
// lies in LDS as it lies in memory, in 16-byte chunks:
//
//  * summed index contiguous ("along"): [row][kDeep], 8 chunks per row; chunk
//    c of row r stands at c ^ swz(r), so that 16 rows read at one chunk
//    column fall on distinct banks;
//  * row index contiguous ("across"): [kDeep][rows].  The 16-bit types read
//    fragments with the transposing LDS load (16 lanes fetch a 4 x 16 block and
//    each gets one column of it); chunk pairs are permuted by the k row so
//    that the 8 k rows a half-wave touches fall on distinct banks.  binary32
//    reads up to 4 neighbouring rows' values per lane at once and gives them to
//    as many fragments: fragment v of a group of V covers rows V*i + v.
//
// Matrix instruction: v_mfma_f32_16x16x32_{bf16,f16} (lane l: row l%16, k =
// 8*(l/16) + 0..7) and v_mfma_f32_16x16x4_f32 (row l%16, k = l/16; the s-th of four
// instructions takes k = 4*(l/16) + s).  The second operand's fragment is passed first, so
// that a lane's four results of a 16 x 16 block are four neighbouring columns of
// one row: D(m = l%16, n = 4*(l/16) + r), and stores are 8 or 16 bytes wide.
#ifndef GEMM_F32_ROWS_TILE_H
#define GEMM_F32_ROWS_TILE_H

#include "rows_common.h"

namespace rows {

template <class E>
constexpr int deep() { return 128 / E::kBytes; }

__device__ inline int swz_along(int r) { return (r ^ (r >> 3)) & 7; }

// Chunk permutation of k row k of an "across" panel of RN rows (16-bit types).
template <int RN>
__device__ inline int swz_across(int k)
{
    if constexpr (RN >= 128)
        return ((k & 3) | ((k >> 3) & 1) << 2) << 1;
    else if constexpr (RN == 64)
        return (((k >> 1) & 1) | ((k >> 3) & 1) << 1) << 1;
    else
        return 0;
}

// LDS element offset of chunk c of row r (along) or of k row r (across).
template <class E, bool ALONG, int RN>
__device__ inline int lds_chunk(int r, int c)
{
    if constexpr (ALONG)
        return r * deep<E>() + (c ^ swz_along(r)) * E::kChunk;
    else if constexpr (E::kBytes == 2)
        return r * RN + (c ^ swz_across<RN>(r)) * E::kChunk;
    else
        return r * RN + c * E::kChunk;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

template <class T>
using lds_ptr = __attribute__((address_space(3))) T *;

// Fragments of F consecutive 16-row blocks from row `row0` of a panel, one
// k step (a step: 32 k of a 16-bit type, 16 of binary32; panels hold two).
template <class E, bool ALONG, int RN, int F>
struct Fragments {
    using T = typename E::T;
    // rows a group of fragments read together covers, /16
    static constexpr int kV = E::kBytes == 2 || ALONG ? 1 : F % 4 == 0 ? 4 : F % 2 == 0 ? 2 : 1;
    u32x4 q[F];      // 8 16-bit values, or 4 binary32 (k = 4*(l/16) + 0..3)

    __device__ inline void read(const T *panel, int row0, int step, int lane)
    {
        const int i = lane % 16, h = lane / 16;
        if constexpr (ALONG) {
#pragma unroll
            for (int f = 0; f < F; ++f)
                q[f] = *reinterpret_cast<const u32x4 *>(panel + lds_chunk<E, true, RN>(row0 + 16 * f + i, 4 * step + h));
        } else if constexpr (E::kBytes == 2) {
            const int k = 32 * step + 8 * h + i / 4;     // this lane's row of the 4 x 16 block
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int col = row0 + 16 * f + 4 * (i % 4);
                const T *p0 = panel + lds_chunk<E, false, RN>(k, col / 8) + col % 8;
                const T *p1 = panel + lds_chunk<E, false, RN>(k + 4, col / 8) + col % 8;
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr<s16x4>)p0);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr<s16x4>)p1);
                q[f] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const T *p = panel + (16 * step + 4 * h + s) * RN + row0 + kV * i;
#pragma unroll
                for (int f = 0; f < F; f += kV) {
                    float v[kV];
                    __builtin_memcpy(v, __builtin_assume_aligned(p + 16 * f, 4 * kV), 4 * kV);
#pragma unroll
                    for (int u = 0; u < kV; ++u)
                        q[f + u][s] = __float_as_uint(v[u]);
                }
            }
        }
    }

    // Row of fragment f's index i (0..15), from row0.
    static __device__ inline int row_of(int f, int i) { return (f / kV) * 16 * kV + kV * i + f % kV; }
};

// d += a . b of one 16 x 16 block and one k step; see the top for the order.
template <class E>
__device__ inline f32x4 mfma_step(u32x4 b, u32x4 a, f32x4 d)
{
    if constexpr (E::kBytes == 4) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            d = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[s]), __uint_as_float(a[s]), d, 0, 0, 0);
        return d;
    } else if constexpr (std::is_same<E, Bf16>::value) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), d, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), d, 0, 0, 0);
    }
}

// A workgroup's BM x BN tile, WM x WN waves of (BM/WM) x (BN/WN).
template <class E, bool A_ALONG, bool B_ALONG, int BM_, int BN_, int WM_, int WN_>
struct Tile {
    using T = typename E::T;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = WM * WN * kWave;
    static constexpr int kFm = BM / WM / 16, kFn = BN / WN / 16;
    static constexpr int kLdsA = BM * deep<E>(), kLdsB = BN * deep<E>();   // elements of a panel
    using Fa = Fragments<E, A_ALONG, BM, kFm>;
    using Fb = Fragments<E, B_ALONG, BN, kFn>;
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "wave tile");

    f32x4 acc[kFm][kFn];

    __device__ inline void clear()
    {
#pragma unroll
        for (int m = 0; m < kFm; ++m)
#pragma unroll
            for (int n = 0; n < kFn; ++n)
                acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    __device__ inline void panel(const T *la, const T *lb, int wm, int wn, int lane)
    {
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            Fa a;
            Fb b;
            a.read(la, wm * (BM / WM), step, lane);
            b.read(lb, wn * (BN / WN), step, lane);
#pragma unroll
            for (int m = 0; m < kFm; ++m)
#pragma unroll
                for (int n = 0; n < kFn; ++n)
                    acc[m][n] = mfma_step<E>(b.q[n], a.q[m], acc[m][n]);
        }
    }

    // f(row, column, 4 neighbouring columns' sums) over the lane's results,
    // row and column within the tile.
    template <class Fn>
    __device__ inline void each(int wm, int wn, int lane, Fn &&f) const
    {
        const int i = lane % 16, h = lane / 16;
        constexpr int V = Fb::kV;
#pragma unroll
        for (int m = 0; m < kFm; ++m) {
            const int row = wm * (BM / WM) + Fa::row_of(m, i);
#pragma unroll
            for (int n = 0; n < kFn; n += V) {
                if constexpr (V == 4) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        f(row, wn * (BN / WN) + Fb::row_of(n, 4 * h + r),
                          f32x4{acc[m][n][r], acc[m][n + 1][r], acc[m][n + 2][r], acc[m][n + 3][r]});
                } else if constexpr (V == 2) {
#pragma unroll
                    for (int r = 0; r < 4; r += 2)
                        f(row, wn * (BN / WN) + Fb::row_of(n, 4 * h + r),
                          f32x4{acc[m][n][r], acc[m][n + 1][r], acc[m][n][r + 1], acc[m][n + 1][r + 1]});
                } else {
                    f(row, wn * (BN / WN) + Fb::row_of(n, 4 * h), acc[m][n]);
                }
            }
        }
    }
};

// Four sums to four neighbouring elements of a row with `left` of them.
template <class E, bool VEC>
__device__ inline void store4(typename E::T *p, f32x4 v, int64_t left)
{
    struct alignas(VEC ? 4 * E::kBytes : E::kBytes) Four {
        typename E::T e[4];
    } o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o.e[i] = (typename E::T)v[i];
    if (left >= 4) {
        __builtin_memcpy(__builtin_assume_aligned(p, alignof(Four)), &o, sizeof o);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left)
                p[i] = o.e[i];
    }
}

// ---------------------------------------------------------------------------
// Where a thread's chunks of a panel come from.  Chunk i of thread tid is the
// panel's 16-byte LDS slot tid + i * threads; at() gives its address for
// the panel that starts at k0 and how many elements of its row there are from there on
// (none: the chunk is zero).
// ---------------------------------------------------------------------------
template <class E, int RN, int NT>
struct Along {
    using T = typename E::T;
    static constexpr bool kAlong = true;
    static constexpr int kSlots = RN * 8, kCount = (kSlots + NT - 1) / NT;
    const T *p[kCount];                              // chunk's address at k0 = 0
    int left[kCount];                                // elements from there on

    // row(r): the panel's row r, NULL if there is none; K elements long.
    template <class Row>
    __device__ inline Along(int tid, int K, Row &&row)
    {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int slot = tid + i * NT, r = slot / 8;
            const int k = (slot % 8 ^ swz_along(r)) * E::kChunk;
            const T *base = kSlots % NT == 0 || slot < kSlots ? row(r) : nullptr;
            p[i] = base != nullptr ? base + k : nullptr;
            left[i] = base != nullptr ? K - k : 0;
        }
    }
    __device__ inline const T *at(int i, int k0, int &n) const
    {
        n = left[i] - k0;
        return p[i] + k0;
    }
};

template <class E, int RN, int NT, class Row>
struct Across {
    using T = typename E::T;
    static constexpr bool kAlong = false;
    static constexpr int kSlots = RN * 8, kCount = (kSlots + NT - 1) / NT;
    static constexpr int kPer = RN / E::kChunk;      // chunks of a k row
    Row row;                                         // row(k): k row k, NULL if there is none
    int tid, K, first, cols;                         // columns first .. of cols

    __device__ inline Across(int tid_, int K_, int first_, int cols_, Row row_)
        : row(row_), tid(tid_), K(K_), first(first_), cols(cols_)
    {
    }
    __device__ inline const T *at(int i, int k0, int &n) const
    {
        const int slot = tid + i * NT, r = slot / kPer;
        int c = slot % kPer;
        if constexpr (E::kBytes == 2)
            c ^= swz_across<RN>(r);
        const int col = first + c * E::kChunk;
        const bool there = (kSlots % NT == 0 || slot < kSlots) && k0 + r < K;
        const T *base = there ? row(k0 + r) : nullptr;
        n = base != nullptr ? cols - col : 0;
        return base + col;
    }
};

template <class E, int RN, int NT, class Row>
__device__ inline Across<E, RN, NT, Row> across(int tid, int K, int first, int cols, Row row)
{
    return Across<E, RN, NT, Row>(tid, K, first, cols, row);
}

// Adds the K-long sums of the tile from panels staged through registers: two
// LDS buffers, one barrier per panel, the next panel's loads in flight
// during a panel's matrix instructions.  lds: 2 * (kLdsA + kLdsB) elements.
template <class E, bool VEC, class Ti, class SrcA, class SrcB>
__device__ inline void sum_panels(Ti &tile, int K, const SrcA &a, const SrcB &b, typename E::T *lds, int tid, int wm,
                                  int wn)
{
    using T = typename E::T;
    constexpr int BK = deep<E>(), NT = Ti::kThreads;
    const int lane = tid % kWave;
    u32x4 ra[SrcA::kCount], rb[SrcB::kCount];
    auto fetch = [&](int k0) {
        int n;
#pragma unroll
        for (int i = 0; i < SrcA::kCount; ++i) {
            const T *p = a.at(i, k0, n);
            ra[i] = load_chunk<E, VEC>(p, n);
        }
#pragma unroll
        for (int i = 0; i < SrcB::kCount; ++i) {
            const T *p = b.at(i, k0, n);
            rb[i] = load_chunk<E, VEC>(p, n);
        }
    };
    auto put = [&](T *panel, int slots, int i, u32x4 v) {
        if (slots % NT == 0 || tid + i * NT < slots)
            *reinterpret_cast<u32x4 *>(panel + (tid + i * NT) * E::kChunk) = v;
    };
    if (K > 0)
        fetch(0);
    int buf = 0;
    for (int k0 = 0; k0 < K; k0 += BK, buf ^= 1) {
        T *la = lds + buf * (Ti::kLdsA + Ti::kLdsB), *lb = la + Ti::kLdsA;
#pragma unroll
        for (int i = 0; i < SrcA::kCount; ++i)
            put(la, SrcA::kSlots, i, ra[i]);
#pragma unroll
        for (int i = 0; i < SrcB::kCount; ++i)
            put(lb, SrcB::kSlots, i, rb[i]);
        __syncthreads();         // the other buffer's readers passed the last one
        if (k0 + BK < K)
            fetch(k0 + BK);
        tile.panel(la, lb, wm, wn, lane);
    }
}

}  // namespace rows

#endif
