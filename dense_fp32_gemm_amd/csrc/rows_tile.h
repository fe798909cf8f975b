// One output tile of a product on the matrix cores, from panels in LDS.
//
// Panels are kDeep16 16-byte chunks (128 bytes) deep in the summed index, kDeep
// elements.  An operand lies in LDS as it lies in memory:
//
//  * summed index contiguous ("along"): [row][kDeep], eight chunks per row; chunk
//    c of row r stands at c ^ swz(r), so that 16 rows read at one chunk
//    column fall on distinct banks;
//  * row index contiguous ("across"): [kDeep][rows].  The 16-bit types read
//    fragments with the transposing LDS load (16 lanes fetch a 4 x 16 block and
//    each gets one column of it); chunk pairs are permuted by the k row so
//    that the 8 k rows a half-wave touches fall on distinct banks.  binary32
//    reads up to 4 neighbouring rows' values per lane at once and gives them to
//    as many fragments: fragment v of a group of V covers rows V*i + v.
//
// Matrix instruction: v_mfma_i32_16x16x64_i8 (lane l: row l%16, k = 16*(l/16) + 0..15),
// v_mfma_f32_16x16x32_{bf16,f16} (k = 8*(l/16) + 0..7) and v_mfma_f32_16x16x4_f32 (row l%16, k = l/16; the s-th of four
// instructions takes k = 4*(l/16) + s).  The second operand's fragment is passed first, so
// that a lane's four results of a 16 x 16 block are four neighbouring columns of
// one row: D(m = l%16, n = 4*(l/16) + r), and stores are 8 or 16 bytes wide.
#ifndef GEMM_F32_ROWS_TILE_H
#define GEMM_F32_ROWS_TILE_H

#include <type_traits>

#include "rows_common.h"

namespace rows {

constexpr int kDeep16 = 8;                           // 16-byte chunks of a panel in the summed index

// Chunk permutation of row r of an "along" panel.  A 128-bit LDS read serves lanes
// {0-3, 12-15, 20-27} together, then {4-11, 16-19, 28-31}, and the same 32
// further: rows 0-3 and 12-15 of one chunk column with rows 4-11 of the next.
// The permutation puts those 16 chunks on the 16 distinct quarters of the 256
// bytes that the banks span.
__device__ inline int swz_along(int r) { return (r >> 1) & 7; }

// Chunk permutation of k row k of an "across" panel of RN rows (16-bit types).  Narrower
// panels than 64 rows have none (the adapters' down-projection of 32 ranks: 40 % of its LDS cycles are
// conflicts, of a kernel of 11 us).
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
        return (r * kDeep16 + (c ^ swz_along(r))) * E::kChunk;
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
// k step (64 k of 8 bits, 32 of a 16-bit type, 16 of binary32: four chunks).
template <class E, bool ALONG, int RN, int F>
struct Fragments {
    using T = typename E::T;
    // rows a group of fragments read together covers, /16
    static constexpr int kV = E::kBytes == 2 || ALONG ? 1 : F % 4 == 0 ? 4 : F % 2 == 0 ? 2 : 1;
    static constexpr int kReads = ALONG ? F : E::kBytes == 2 ? 2 * F : 4 * F / kV;   // LDS instructions
    u32x4 q[F];      // 16 8-bit values, 8 16-bit ones, or 4 binary32 (k = 4*(l/16) + 0..3)

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

// Four sums of a lane: binary32, or whole numbers of the 8-bit products.
template <class E>
using Sum4 = std::conditional_t<E::kBytes == 1, i32x4, f32x4>;

// d += a . b of one 16 x 16 block and the s-th instruction of a k step (kPerStep
// of them); see the top for the order.
template <class E>
constexpr int kPerStep = E::kBytes == 4 ? 4 : 1;
template <class E>
__device__ inline Sum4<E> mfma(u32x4 b, u32x4 a, Sum4<E> d, int s)
{
    if constexpr (E::kBytes == 1)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), d, 0, 0, 0);
    else if constexpr (E::kBytes == 4)
        return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[s]), __uint_as_float(a[s]), d, 0, 0, 0);
    else if constexpr (std::is_same<E, Bf16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), d, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), d, 0, 0, 0);
}

// A workgroup's BM x BN tile, WM x WN waves of (BM/WM) x (BN/WN).
template <class E, bool A_ALONG, bool B_ALONG, int BM_, int BN_, int WM_, int WN_>
struct Tile {
    using T = typename E::T;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = WM * WN * kWave;
    static constexpr int kFm = BM / WM / 16, kFn = BN / WN / 16;
    static constexpr int kDeep = kDeep16 * E::kChunk, kSteps = kDeep16 / 4;
    static constexpr int kMfma = kFm * kFn * kPerStep<E>;                 // matrix instructions of a step
    static constexpr int kLdsA = BM * kDeep, kLdsB = BN * kDeep;           // elements of a panel
    using Fa = Fragments<E, A_ALONG, BM, kFm>;
    using Fb = Fragments<E, B_ALONG, BN, kFn>;
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "wave tile");
    static_assert((A_ALONG || (BM & (BM - 1)) == 0) && (B_ALONG || (BN & (BN - 1)) == 0),
                  "the chunk permutations across rows are made for powers of two");

    Sum4<E> acc[kFm][kFn];

    __device__ inline void clear()
    {
#pragma unroll
        for (int m = 0; m < kFm; ++m)
#pragma unroll
            for (int n = 0; n < kFn; ++n)
                acc[m][n] = Sum4<E>{0, 0, 0, 0};
    }

    // One step's fragments of a panel.
    struct Step {
        Fa a;
        Fb b;
        __device__ inline void read(const T *panel, int step, int wm, int wn, int lane)
        {
            a.read(panel, wm * (BM / WM), step, lane);
            b.read(panel + kLdsA, wn * (BN / WN), step, lane);
        }
    };

    __device__ inline void multiply(const Step &s)
    {
        // block by block within an instruction of the step: neighbouring
        // instructions do not wait for one another's sums
#pragma unroll
        for (int i = 0; i < kPerStep<E>; ++i)
#pragma unroll
            for (int m = 0; m < kFm; ++m)
#pragma unroll
                for (int n = 0; n < kFn; ++n)
                    acc[m][n] = mfma<E>(s.b.q[n], s.a.q[m], acc[m][n], i);
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

// Four sums to four neighbouring elements of a row with `left` of them (VEC: at least four).
template <class E, bool VEC>
__device__ inline void store4(typename E::T *p, f32x4 v, int64_t left)
{
    struct alignas(VEC ? 4 * E::kBytes : E::kBytes) Four {
        typename E::T e[4];
    } o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o.e[i] = (typename E::T)v[i];
    if (VEC || left >= 4) {
        __builtin_memcpy(__builtin_assume_aligned(p, alignof(Four)), &o, sizeof o);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left)
                p[i] = o.e[i];
    }
}

// Debug build (-DGEMM_F32_POISON_LDS): every LDS slot that a panel's load is about to fill is
// first set to NaN of whichever type by the wave that issues the load, so that a read
// before the panel has landed, or of a buffer that is being refilled, carries NaN into the result
// instead of older numbers.
#ifdef GEMM_F32_POISON_LDS
constexpr bool kPoisonLds = true;
#else
constexpr bool kPoisonLds = false;
#endif
__device__ inline void poison16(void *p) { *reinterpret_cast<u32x4 *>(p) = u32x4{~0u, ~0u, ~0u, ~0u}; }

// ---------------------------------------------------------------------------
// Where a thread's chunks of a panel come from.  Chunk i of thread tid is the
// panel's 16-byte LDS slot tid + i * threads.  base is a uniform address, p[i]
// (Along) or row(k) (Across) lies a byte offset off it, kNowhere: zeros.
// ---------------------------------------------------------------------------
constexpr uint32_t kNowhere = 0x80000000u;           // a buffer offset that reads as 0
constexpr int kRawBufferFlags = 0x00020000;          // dword 3 of a raw buffer resource

// A pointer that is the same in all lanes, in scalar registers (the compiler
// does not always see it, and loops over lanes around every load then).
__device__ inline const char *uniform(const void *p)
{
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u), hi = __builtin_amdgcn_readfirstlane((int)(u >> 32));
    return (const char *)((uint64_t)hi << 32 | lo);
}

// `bytes` as a buffer's size: loads past it give zeros, and so does kNowhere.
__device__ inline uint32_t buffer_size(int64_t bytes)
{
    return (uint32_t)(bytes < 0 ? 0 : bytes < (int64_t)kNowhere ? bytes : (int64_t)kNowhere);
}

// Operand rows contiguous in the summed index.  row(i, r): byte offset from base of the
// panel's row r (of chunk i), negative if there is none; rows are K elements long.
template <class E, int RN, int NT>
struct Along {
    using T = typename E::T;
    static constexpr bool kListed = false;
    static constexpr int kSlots = RN * kDeep16, kDeep = kDeep16 * E::kChunk, kCount = (kSlots + NT - 1) / NT;
    const char *base;
    int64_t off[kCount];
    int64_t ld;                                      // bytes between rows
    int K, tid, rows;                                // rows: from base on

    static constexpr bool kAlong = true, kOneColumn = false;
    // Bytes from base to the operand's end, in whole dwords: the last chunk of a row that is no
    // whole number of chunks long reads what follows (and is cleared in LDS), zeros past the end.
    __device__ inline int64_t extent() const { return ((rows - 1) * ld + (int64_t)K * E::kBytes + 3) / 4 * 4; }
    // Panel row of chunk i.
    static __device__ inline int row_of(int i, int tid) { return (tid + i * NT) / kDeep16; }

    template <class Row>
    __device__ inline Along(const T *base_, int tid_, int K_, int64_t ld_, int rows_, Row &&row)
        : base(uniform(base_)), ld(ld_ * E::kBytes), K(__builtin_amdgcn_readfirstlane(K_)), tid(tid_), rows(rows_)
    {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int slot = tid + i * NT, r = slot / kDeep16;
            const int64_t o = kSlots % NT == 0 || slot < kSlots ? row(i, r) : -1;
            off[i] = o < 0 ? -1 : o + first_k(i) * E::kBytes;
        }
    }
    __device__ inline int64_t step() const { return kDeep * E::kBytes; }   // bytes from panel to panel
    // Whether the panel at k0 is the last: chunks that panel 0 has may be missing from it,
    // and others reach past a row's end.
    __device__ inline bool last(int k0) const { return K - k0 <= kDeep; }
    // First k of chunk i in panel 0.  (Recomputed where it is needed: registers are short.)
    __device__ inline int first_k(int i) const
    {
        const int slot = tid + i * NT;
        return (slot % kDeep16 ^ swz_along(slot / kDeep16)) * E::kChunk;
    }
    // Elements from chunk i of the panel at k0 to its row's end (none: zeros), and its
    // offset; inside() for a row that is there.
    __device__ inline int inside(int i, int k0) const { return K - k0 - first_k(i); }
    __device__ inline int left(int i, int k0) const { return off[i] < 0 ? 0 : inside(i, k0); }
    __device__ inline int64_t offset(int i, int) const { return off[i]; }
};

// Operand rows contiguous across the summed index: K of them, ld elements apart, columns
// first .. of cols.
template <class E, int RN, int NT>
struct Across {
    using T = typename E::T;
    static constexpr bool kListed = false;
    static constexpr int kSlots = RN * kDeep16, kDeep = kDeep16 * E::kChunk, kCount = (kSlots + NT - 1) / NT;
    static constexpr int kPer = RN / E::kChunk;      // chunks of a k row
    const char *base;
    int64_t ld;                                      // bytes between k rows
    int tid, K, first, cols;
    int rows;                                        // from base on

    __device__ inline Across(const T *base_, int tid_, int K_, int64_t ld_, int first_, int cols_, int rows_)
        : base(uniform(base_)), ld(ld_ * E::kBytes), tid(tid_), K(__builtin_amdgcn_readfirstlane(K_)), first(first_),
          cols(cols_), rows(rows_)
    {
    }
    __device__ inline Across(const T *base_, int tid_, int K_, int64_t ld_, int first_, int cols_)
        : Across(base_, tid_, K_, ld_, first_, cols_, K_)
    {
    }
    static constexpr bool kAlong = false;
    // Bytes from base to the operand's end, in whole dwords: a chunk that crosses the last
    // row's end reads zeros there (one that crosses another row's end reads the
    // next row's start, for columns that are not stored).
    __device__ inline int64_t extent() const { return ((rows - 1) * ld + (int64_t)cols * E::kBytes + 3) / 4 * 4; }
    // A thread's chunks are kRowStep k rows apart, and mostly in one column: the chunk
    // permutation depends on k's bits 0, 1 and 3 only.
    static constexpr int kRowStep = NT / kPer;
    static constexpr bool kOneColumn = E::kBytes == 4 || RN < 64 || kRowStep % 16 == 0 || kCount == 1;
    static_assert(NT % kPer == 0, "a thread's chunks keep their place in the k row");
    __device__ inline int krow(int i) const { return tid / kPer + i * kRowStep; }
    __device__ inline int col(int i) const
    {
        int c = tid % kPer;
        if constexpr (E::kBytes == 2)
            c ^= swz_across<RN>(krow(kOneColumn ? 0 : i));
        return first + c * E::kChunk;
    }
    // k rows from chunk 0 to chunk i, as loaded.
    static __device__ inline int row_step(int i) { return i * kRowStep; }
    __device__ inline int64_t step() const { return kDeep * ld; }
    // Whether k rows may be missing from the panel at k0, or a chunk of it (of kChunk k rows
    // where they are one element long) reaches past the last one.
    __device__ inline bool last(int k0) const { return K - k0 <= kDeep + E::kChunk; }
    __device__ inline int left(int i, int k0) const
    {
        return (kSlots % NT == 0 || tid + i * NT < kSlots) && k0 + krow(i) < K ? cols - col(i) : 0;
    }
    __device__ inline int inside(int i, int k0) const { return left(i, k0); }
    __device__ inline int64_t offset(int i, int) const { return krow(i) * ld + (int64_t)col(i) * E::kBytes; }
};

// The same with k rows in any order: k row k is row list[k] / per_row of
// `rows` (negative or past them: zeros).  The direct loads take the rows' offsets
// from LDS, where refill() puts kBlock of them at a time.
template <class E, int RN, int NT>
struct Gathered : Across<E, RN, NT> {
    using Base = Across<E, RN, NT>;
    static constexpr int kBlock = 512;
    static constexpr bool kListed = true;
    const int *list;                                 // NULL: k itself
    uint32_t *ahead;                                 // LDS: 2 * kBlock offsets
    Divisor per_row;
    __device__ inline Gathered(const typename E::T *base_, int tid_, int K_, int64_t ld_, int first_, int cols_,
                               const int *list_, Divisor per_row_, int rows_, uint32_t *ahead_)
        : Base(base_, tid_, K_, ld_, first_, cols_, rows_), list(list_), ahead(ahead_), per_row(per_row_)
    {
    }
    __device__ inline int row(int k) const
    {
        const int s = list != nullptr ? list[k] : k, r = per_row.of(s);
        return s < 0 || r >= this->rows ? -1 : r;
    }
    __device__ inline int64_t step() const { return 0; }
    __device__ inline int left(int i, int k0) const
    {
        const int n = Base::left(i, k0);
        return n > 0 && row(k0 + this->krow(i)) >= 0 ? n : 0;
    }
    __device__ inline int64_t offset(int i, int k0) const
    {
        return row(k0 + this->krow(i)) * this->ld + (int64_t)this->col(i) * E::kBytes;
    }
    // Called by every thread before the barrier ahead of the panel at k0's loads.
    __device__ inline void refill(int k0) const
    {
        if (k0 % kBlock != 0)
            return;
        for (int j = this->tid; j < kBlock; j += NT) {
            const int k = k0 + j, r = k < this->K ? row(k) : -1;
            ahead[(k0 / kBlock % 2) * kBlock + j] = r < 0 ? kNowhere : (uint32_t)(r * this->ld);
        }
    }
};

// ---------------------------------------------------------------------------
// The K loop: adds the K-long sums to the (cleared) tile.
//
// DMA: buffer loads write panels straight into a ring of S LDS buffers of
// kLdsA + kLdsB elements, up to S panels ahead of the matrix cores, one
// barrier per panel; fragments are read half a panel before they are
// multiplied.  For rows on 4-byte boundaries less than 2^31 bytes from
// their base.  Else the chunks are staged through registers into two
// buffers, element by element at a row's end.
// ---------------------------------------------------------------------------
// Between a group's writes to LDS and its reads of them: a barrier, or only program
// order where the group is one wave (whose LDS accesses are in order).
template <int NT>
__device__ inline void group_sync()
{
    if constexpr (NT > kWave)
        __syncthreads();
    else
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// binary32 sums (FOLD) are taken kFold k at a time and the parts then added up: rounding errors
// grow with the length of a chain of additions.  128 rows over 8 groups, K = 4096, N = 512: root mean square
// error 4.1e-7 of the result's, 11.4e-7 in one chain.  us with and without: those rows with N = 1024
// 58.0 and 59.0; 4096 rows, 2048 x 2048: 281.6 and 280.7, both gradients 573.6 and 568.3; adapters,
// 2050 rows, 4096 x 4096: 576 and 572.  Not where K is split over workgroups anyway (the adapters'
// few rows and down-projection, 94 and 84 for 400 rows, 4096 x 2048), and not for the 16-bit types, whose
// results are rounded to fewer bits than the longest chain here loses.
constexpr int kFold = 512;
template <class E, class Ti, bool FOLD>
struct Parts {
    static constexpr bool kUsed = FOLD && E::kBytes == 4;
    f32x4 sum[kUsed ? Ti::kFm : 1][kUsed ? Ti::kFn : 1];
    __device__ inline void clear()
    {
        if constexpr (kUsed)
#pragma unroll
            for (int m = 0; m < Ti::kFm; ++m)
#pragma unroll
                for (int n = 0; n < Ti::kFn; ++n)
                    sum[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ inline void fold(Ti &tile)
    {
        if constexpr (kUsed)
#pragma unroll
            for (int m = 0; m < Ti::kFm; ++m)
#pragma unroll
                for (int n = 0; n < Ti::kFn; ++n) {
                    sum[m][n] += tile.acc[m][n];
                    tile.acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
    }
    __device__ inline void finish(Ti &tile)
    {
        if constexpr (kUsed)
#pragma unroll
            for (int m = 0; m < Ti::kFm; ++m)
#pragma unroll
                for (int n = 0; n < Ti::kFn; ++n)
                    tile.acc[m][n] += sum[m][n];
    }
};

template <class E, bool FOLD, class Ti, class SrcA, class SrcB>
__device__ inline void sum_panels_staged(Ti &tile, int K, const SrcA &a, const SrcB &b, typename E::T *lds, int tid,
                                         int wm, int wn)
{
    using T = typename E::T;
    constexpr int BK = Ti::kDeep, NT = Ti::kThreads;
    const int lane = tid % kWave;
    u32x4 ra[SrcA::kCount], rb[SrcB::kCount];
    auto load = [&](const auto &src, int i, int k0) {
        const int n = src.left(i, k0);
        const char *p = src.base + (int64_t)(k0 / BK) * src.step();
        return load_chunk<E, false>((const T *)(p + (n > 0 ? src.offset(i, k0) : 0)), n);
    };
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < SrcA::kCount; ++i)
            ra[i] = load(a, i, k0);
#pragma unroll
        for (int i = 0; i < SrcB::kCount; ++i)
            rb[i] = load(b, i, k0);
    };
    auto put = [&](T *panel, int slots, int i, u32x4 v) {
        if (slots % NT == 0 || tid + i * NT < slots)
            *reinterpret_cast<u32x4 *>(panel + (tid + i * NT) * E::kChunk) = v;
    };
    // Poisoned: before the barrier that readers of a panel wait at, all of it and then its data,
    // so that what is not written before the barrier, or by nobody, is NaN.
    auto poison = [&](T *panel) {
        if constexpr (kPoisonLds) {
            for (int c = tid; c < (Ti::kLdsA + Ti::kLdsB) / E::kChunk; c += NT)
                poison16(panel + c * E::kChunk);
            group_sync<NT>();
        }
    };
    Parts<E, Ti, FOLD> parts;
    parts.clear();
    if (K > 0)
        fetch(0);
    int buf = 0;
    for (int k0 = 0; k0 < K; k0 += BK, buf ^= 1) {
        T *la = lds + buf * (Ti::kLdsA + Ti::kLdsB), *lb = la + Ti::kLdsA;
        poison(la);
#pragma unroll
        for (int i = 0; i < SrcA::kCount; ++i)
            put(la, SrcA::kSlots, i, ra[i]);
#pragma unroll
        for (int i = 0; i < SrcB::kCount; ++i)
            put(lb, SrcB::kSlots, i, rb[i]);
        group_sync<NT>();        // the other buffer's readers passed the last one
        if (k0 + BK < K)
            fetch(k0 + BK);
        if (parts.kUsed && k0 % kFold == 0)
            parts.fold(tile);
#pragma unroll
        for (int step = 0; step < Ti::kSteps; ++step) {
            typename Ti::Step f;
            f.read(la, step, wm, wn, lane);
            tile.multiply(f);
        }
    }
    parts.finish(tile);
}

// NaN over the slots of a panel that the wave's loads will fill (poisoned build).
template <class Src, class E, int NT>
__device__ inline void poison_slots(typename E::T *panel, int wave)
{
    if constexpr (kPoisonLds) {
#pragma unroll
        for (int i = 0; i < Src::kCount; ++i)
            if (Src::kSlots % NT == 0 || i * NT + wave * kWave < Src::kSlots)
                poison16(panel + (i * NT + wave * kWave + (int)(threadIdx.x % kWave)) * E::kChunk);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// The panel loads of one operand by one wave: lane l's 16 bytes land at the
// wave's LDS base + 16 * l.  Offsets that differ by whole rows are one register.
// fire() takes the panels one after the other, from the one at `from` on.
template <class E, class Src, int NT>
struct PanelLoads {
    static_assert(Src::kSlots % kWave == 0, "whole waves");
    using T = typename E::T;
    static constexpr bool kOne = Src::kOneColumn;
    uint32_t off[kOne ? 1 : Src::kCount];
    const char *base;                                // of the next panel
    int64_t step;                                    // to the panel after it
    __device__ inline PanelLoads(const Src &src, int from = 0) : step(src.step())
    {
        base = src.base + from / Src::kDeep * step;
        if constexpr (kOne) {
            off[0] = src.col(0) < src.cols ? (uint32_t)src.offset(0, 0) : kNowhere;
        } else {
#pragma unroll
            for (int i = 0; i < Src::kCount; ++i)
                off[i] = src.left(i, 0) > 0 ? (uint32_t)src.offset(i, 0) : kNowhere;
        }
    }
    // Past kNowhere, where that is what off[0] is: rows span less than 2^31 bytes.
    __device__ inline uint32_t at(const Src &src, int i) const
    {
        if constexpr (!kOne)
            return off[i];
        else
            return off[0] + (uint32_t)Src::row_step(i) * (uint32_t)src.ld;
    }
    __device__ inline void fire(const Src &src, int k0, T *panel, int wave)
    {
        auto load = [&](uint32_t size, int i, uint32_t o) {
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)size, kRawBufferFlags);
            if (Src::kSlots % NT != 0 && (i * NT + wave * kWave) >= Src::kSlots)
                return;                              // whole waves: kSlots is a multiple of 64
            auto *dst = (lds_ptr<void>)(panel + (i * NT + wave * kWave) * E::kChunk);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst, 16, o, 0, 0, 0);
        };
        poison_slots<Src, E, NT>(panel, wave);
        // The operand's end and missing chunks matter to its last panel alone (last()).
        if (!src.last(k0)) {
#pragma unroll
            for (int i = 0; i < Src::kCount; ++i)
                load(kNowhere, i, at(src, i));
        } else {
            const uint32_t size = buffer_size(src.extent() - (base - src.base));
#pragma unroll
            for (int i = 0; i < Src::kCount; ++i)
                load(size, i, src.inside(i, k0) > 0 ? at(src, i) : kNowhere);
        }
        base += step;
    }
};

template <class E, int RN, int NT>
struct PanelLoads<E, Gathered<E, RN, NT>, NT> {
    using Src = Gathered<E, RN, NT>;
    using T = typename E::T;
    __device__ inline PanelLoads(const Src &) {}
    __device__ inline void fire(const Src &src, int k0, T *panel, int wave)
    {
        static_assert(Src::kSlots % NT == 0 && Src::kBlock % Src::kDeep == 0, "whole panels");
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)src.base, 0, (int)buffer_size(src.extent()), kRawBufferFlags);
        static_assert(Src::kOneColumn, "one column a thread");
        const int col = src.col(0);
        poison_slots<Src, E, NT>(panel, wave);
        const uint32_t *block = src.ahead + (k0 / Src::kBlock % 2) * Src::kBlock + k0 % Src::kBlock;
#pragma unroll
        for (int i = 0; i < Src::kCount; ++i) {
            const uint32_t row = block[src.krow(i)];
            const uint32_t o = row == kNowhere || col >= src.cols ? kNowhere : row + col * E::kBytes;
            auto *dst = (lds_ptr<void>)(panel + (i * NT + wave * kWave) * E::kChunk);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst, 16, o, 0, 0, 0);
        }
    }
};

// The panel at k0 of one operand (rows a whole number of chunks long, if along) into LDS,
// complete after the wait and barrier that follow.
template <class E, bool DMA, int NT, class Src>
__device__ inline void load_panel(const Src &src, int k0, typename E::T *panel, int tid)
{
    using T = typename E::T;
    if constexpr (DMA) {
        PanelLoads<E, Src, NT> loads(src, k0);
        loads.fire(src, k0, panel, __builtin_amdgcn_readfirstlane(tid / kWave));
    } else {
        const char *p = src.base + (int64_t)(k0 / Src::kDeep) * src.step();
#pragma unroll
        for (int i = 0; i < Src::kCount; ++i) {
            const int slot = tid + i * NT, n = src.left(i, k0);
            if (Src::kSlots % NT == 0 || slot < Src::kSlots)
                *reinterpret_cast<u32x4 *>(panel + slot * E::kChunk) =
                    load_chunk<E, false>((const T *)(p + (n > 0 ? src.offset(i, k0) : 0)), n);
        }
    }
}

// Zeros over what the last chunk of an "along" operand's rows, K elements long, brought from
// behind them, in the panel at k0 that they end in (K no whole number of chunks).
template <class E, class Src, int RN, int NT>
__device__ inline void clear_tail(const Src &src, int k0, typename E::T *panel, int tid)
{
    if constexpr (Src::kAlong) {
        const int chunk = (src.K - k0) / E::kChunk, from = src.K % E::kChunk;
        if (from == 0)
            return;
        for (int r = tid; r < RN; r += NT) {
            typename E::T *p = panel + lds_chunk<E, true, RN>(r, chunk);
#pragma unroll 1
            for (int e = from; e < E::kChunk; ++e)
                p[e] = (typename E::T)0.f;
        }
    }
}

// Half a panel's work: fragments of one step are read while those of the other
// step, read half a panel ago, are multiplied.  `freed` (what fire() fills) and
// `panel` (what is read) do not overlap; saying so keeps the compiler
// from waiting for the loads in flight before it reads.
template <class E, class Ti, class Fire>
__device__ __forceinline__ void half_panel(Ti &tile, const typename E::T *__restrict__ panel, typename E::T *__restrict__ freed,
                                           Fire &&fire, int step, typename Ti::Step &read, const typename Ti::Step &done,
                                           int wm, int wn, int lane)
{
    fire(freed);
    __builtin_amdgcn_sched_barrier(0);
    read.read(panel, step, wm, wn, lane);
    tile.multiply(done);
    // One LDS read behind each matrix instruction while there are any: issued in a
    // row, the reads of all waves would queue and the matrix cores idle.
    constexpr int kReads = Ti::Fa::kReads + Ti::Fb::kReads, kMfma = Ti::kMfma;
#pragma unroll
    for (int i = 0; i < kReads && i < kMfma - 1; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, kMfma, 0);
    __builtin_amdgcn_sched_barrier(0);
}

// The panel S - 1 ahead is loaded into `freed`, then this one's fragments are
// read and multiplied, the first operand's two row blocks ahead of their use and the
// second's a step: half the fragments' registers (bf16, 16384 places over 8 groups,
// 2048 x 2048, both gradients: 342 us against 356 with a step read, then multiplied).
template <class E, class Ti, class Fire>
__device__ __forceinline__ void whole_panel(Ti &tile, const typename E::T *__restrict__ panel, typename E::T *__restrict__ freed,
                                            Fire &&fire, int wm, int wn, int lane)
{
    fire(freed);
    __builtin_amdgcn_sched_barrier(0);
    static_assert(Ti::kSteps == 2 && kPerStep<E> == 1 && Ti::kFm >= 2, "the order below");
    typename Ti::Step f[2];
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        f[step].b.read(panel + Ti::kLdsA, wn * (Ti::BN / Ti::WN), step, lane);
        f[step].a.read(panel, wm * (Ti::BM / Ti::WM), step, lane);
        tile.multiply(f[step]);
    }
    constexpr int kB = Ti::Fb::kReads, kA = Ti::Fa::kReads / Ti::kFm, kFirst = kB + 2 * kA;   // LDS reads
    __builtin_amdgcn_sched_group_barrier(0x100, kFirst, 0);
#pragma unroll
    for (int step = 0; step < 2; ++step) {
#pragma unroll
        for (int m = 0; m < Ti::kFm - 2; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, Ti::kFn, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kA, 0);
        }
        if (step == 0) {
            __builtin_amdgcn_sched_group_barrier(0x008, Ti::kFn, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kFirst / 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, Ti::kFn, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kFirst - kFirst / 2, 0);
        }
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 2 * Ti::kFn, 0);
    __builtin_amdgcn_sched_barrier(0);
}

template <class E, int S, bool FOLD, class Ti, class SrcA, class SrcB>
__device__ inline void sum_panels_dma(Ti &tile, int K, const SrcA &a, const SrcB &b, typename E::T *lds, int tid,
                                      int wm, int wn)
{
    using T = typename E::T;
    constexpr int BK = Ti::kDeep, NT = Ti::kThreads, kPanel = Ti::kLdsA + Ti::kLdsB;
    // A wave's loads per panel (where the slots are no multiple of the threads the last
    // waves have fewer, and wait for more than they must).
    constexpr int kLoads = SrcA::kSlots / NT + SrcB::kSlots / NT;
    const int lane = tid % kWave, wave = NT == kWave ? 0 : __builtin_amdgcn_readfirstlane(tid / kWave);
    // (An empty sum runs one panel of zeros: a way around the loop would cost a second
    // set of registers for the sums.)
    PanelLoads<E, SrcA, NT> pa(a);
    PanelLoads<E, SrcB, NT> pb(b);
    auto fire = [&](int k0, T *panel) {
        pa.fire(a, k0, panel, wave);
        pb.fire(b, k0, panel + Ti::kLdsA, wave);
    };
    // The panel at k0 (in `panel`) has landed when no more than `after` whole panels
    // behind it are in flight, and every wave's LDS accesses so far are complete.
    auto landed = [&](int k0, T *panel, auto after) {
        if (k0 + (decltype(after)::value + 1) * BK <= K)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(after)::value * kLoads) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        if constexpr (NT > kWave)
            __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if ((SrcA::kAlong || SrcB::kAlong) && K % E::kChunk != 0 && k0 + BK > K) {
            clear_tail<E, SrcA, Ti::BM, NT>(a, k0, panel, tid);
            clear_tail<E, SrcB, Ti::BN, NT>(b, k0, panel + Ti::kLdsA, tid);
            group_sync<NT>();
        }
    };
    if constexpr (SrcA::kListed) {
        a.refill(0);
        __syncthreads();
    }
    // With rows from a list, 16-bit types read two row blocks ahead instead of half a panel: less
    // for the registers, of which a step of fragments ahead took the rest (see whole_panel()).
    if constexpr (SrcA::kListed && E::kBytes == 2) {
#pragma unroll
        for (int q = 0; q < S - 1; ++q)
            if (q == 0 || q * BK < K)
                fire(q * BK, lds + q * kPanel);
        int now = 0, next = S - 1;
        for (int k0 = 0; k0 < K; k0 += BK) {
            if constexpr (SrcA::kListed)
                a.refill(k0 + (S - 1) * BK);
            landed(k0, lds + now * kPanel, std::integral_constant<int, S - 2>{});
            whole_panel<E>(tile, lds + now * kPanel, lds + next * kPanel,
                           [&](T *freed) {
                               if (k0 + (S - 1) * BK < K)
                                   fire(k0 + (S - 1) * BK, freed);
                           },
                           wm, wn, lane);
            now = now + 1 == S ? 0 : now + 1;
            next = next + 1 == S ? 0 : next + 1;
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < S; ++q)
        if (q == 0 || q * BK < K)
            fire(q * BK, lds + q * kPanel);
    typename Ti::Step f0, f1;
    landed(0, lds, std::integral_constant<int, S - 1>{});
    f0.read(lds, 0, wm, wn, lane);
    Parts<E, Ti, FOLD> parts;
    parts.clear();
    int now = 0;
    for (int k0 = BK; k0 < K;) {                     // k0: the panel after this one
        // (a loop around the loop: a test in every panel would cost binary32 products a hundredth)
        const int end = parts.kUsed ? min(K, k0 + kFold) : K;
        for (; k0 < end; k0 += BK) {
            T *panel = lds + now * kPanel;
            half_panel<E>(tile, panel, (T *)nullptr, [](T *) {}, 1, f1, f0, wm, wn, lane);
            if constexpr (SrcA::kListed)
                a.refill(k0 + (S - 1) * BK);
            now = now + 1 == S ? 0 : now + 1;
            landed(k0, lds + now * kPanel, std::integral_constant<int, S - 2>{});
            half_panel<E>(tile, lds + now * kPanel, panel,
                          [&](T *freed) {
                              if (k0 + (S - 1) * BK < K)
                                  fire(k0 + (S - 1) * BK, freed);
                          },
                          0, f0, f1, wm, wn, lane);
        }
        parts.fold(tile);
    }
    half_panel<E>(tile, lds + now * kPanel, (T *)nullptr, [](T *) {}, 1, f1, f0, wm, wn, lane);
    tile.multiply(f1);
    parts.finish(tile);
}

template <class E, bool DMA, int S, bool FOLD = true, class Ti, class SrcA, class SrcB>
__device__ inline void sum_panels(Ti &tile, int K, const SrcA &a, const SrcB &b, typename E::T *lds, int tid, int wm,
                                  int wn)
{
    if constexpr (DMA)
        sum_panels_dma<E, S, FOLD>(tile, K, a, b, lds, tid, wm, wn);
    else
        sum_panels_staged<E, FOLD>(tile, K, a, b, lds, tid, wm, wn);
}

// ---------------------------------------------------------------------------
// Tile numbering
// ---------------------------------------------------------------------------
// Workgroups are dealt to the dies round-robin; renumbered so that each die
// gets a contiguous range of tiles, whose operands its L2 then shares.
__device__ inline int die_contiguous(int w, int total, int xcds)
{
    if (xcds == 8)                                   // a whole MI355X: without divisions
        return (w & 7) * (total >> 3) + min(w & 7, total & 7) + (w >> 3);
    const int per = total / xcds, rem = total % xcds, xcd = w % xcds;
    return xcd * per + (xcd < rem ? xcd : rem) + w / xcds;
}

// Workgroup w's part of `total` tiles on a device that holds `slots` workgroups
// at once: whole tiles while they fill rounds of slots; the tiles of a last
// round that fills at most half (a quarter) of the slots are cut into two (four).
struct Part {
    int tile, cut, piece;    // cut: 1, 2 or 4 pieces; tile < 0: nothing to do
};
__device__ inline Part part_of(int w, int total, int slots, int xcds)
{
    const int whole = total / slots * slots, rest = total - whole;
    if (w < whole)
        return Part{die_contiguous(w, whole, xcds), 1, 0};
    const int cut = 4 * rest <= slots ? 4 : 2 * rest <= slots ? 2 : 1;
    if (w - whole >= rest * cut)
        return Part{-1, 1, 0};
    const int q = die_contiguous(w - whole, rest * cut, xcds);
    return Part{whole + q / cut, cut, q % cut};
}

// Rows that the direct loads can address: on 4-byte boundaries, `span` rows of ld
// elements within 2^31 bytes.
inline bool dma_rows(int type, const void *p, int64_t ld, int64_t span)
{
    const int b = type_bytes(type);
    return aligned_to(p, 4) && ld * b % 4 == 0 && span * ld < (int64_t)kNowhere / b - 16;
}

// Rows that stores of four elements can write.
inline bool vector_rows(int type, const void *p, int64_t ld, int64_t stride, int64_t cols)
{
    return aligned_to(p, 4 * type_bytes(type)) && ld % 4 == 0 && stride % 4 == 0 && cols % 4 == 0;
}

}  // namespace rows

#endif
