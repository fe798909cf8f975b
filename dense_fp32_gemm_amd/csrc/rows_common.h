// Element types, loads and small wave-level helpers of the row-chosen
// products (include/gemm_f32_rows.h).
#ifndef GEMM_F32_ROWS_COMMON_H
#define GEMM_F32_ROWS_COMMON_H

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include "gemm_f32_rows.h"
#include "internal.h"

namespace rows {

constexpr int kWave = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// An element type as the kernels see it: Bytes of storage, Chunk elements in
// 16 bytes, conversions to and from binary32 (to the nearest, ties to even).
struct F32 {
    using T = float;
    static constexpr int kBytes = 4, kChunk = 4;
};
struct Bf16 {
    using T = __bf16;
    static constexpr int kBytes = 2, kChunk = 8;
};
struct F16 {
    using T = _Float16;
    static constexpr int kBytes = 2, kChunk = 8;
};

// 16 bytes of elements.
template <class E>
union Chunk {
    u32x4 raw;
    typename E::T e[E::kChunk];
};

// Calls f(E{}) for the element type `type`; false if there is none.
template <class Fn>
inline bool with_type(int type, Fn &&f)
{
    switch (type) {
    case GEMM_F32_TYPE_F32: f(F32{}); return true;
    case GEMM_F32_TYPE_BF16: f(Bf16{}); return true;
    case GEMM_F32_TYPE_F16: f(F16{}); return true;
    default: return false;
    }
}

inline int type_bytes(int type) { return type == GEMM_F32_TYPE_F32 ? 4 : 2; }
inline bool known_type(int type) { return type >= GEMM_F32_TYPE_F32 && type <= GEMM_F32_TYPE_F16; }
inline bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// The largest of the sizes that kernels count along: loops step past a size by up to a ring of
// panels, a block of row offsets or a workgroup's columns, all under 4096, in 32 bits.
constexpr int kMaxSize = INT32_MAX - 4095;
inline bool bad_size(int n) { return n < 0 || n > kMaxSize; }
inline int at_least_one(int n) { return n > 1 ? n : 1; }

inline int launched() { return hipGetLastError() == hipSuccess ? GEMM_F32_OK : GEMM_F32_ERR_LAUNCH; }

// Division of 0 .. 2^31 - 1 by a number 1 .. 2^31 - 1 known on the host:
// n / d = n * m >> 31 + L with L = ceil(log2 d), m = ceil(2^(31+L) / d).  m d exceeds
// 2^(31+L) by less than d <= 2^L, so the quotient by less than n / 2^31 < 1 /d's share of it.
struct Divisor {
    uint32_t m;
    int shift;
    explicit Divisor(int d)
    {
        int L = 0;
        while (((int64_t)1 << L) < d)
            ++L;
        shift = 31 + L;
        m = (uint32_t)(((((uint64_t)1 << shift) + (uint64_t)d - 1)) / (uint64_t)d);
    }
    __device__ inline int of(int n) const { return (int)((uint64_t)(uint32_t)n * m >> shift); }
};

// 16 bytes of a row that has `left` elements from p on, +0 behind them.
// Global loads of 16 bytes may start at any element of the types here; rows
// that are 16-byte aligned and a whole number of chunks long (VEC) need no
// element-wise tail.
template <class E, bool VEC>
__device__ inline u32x4 load_chunk(const typename E::T *p, int64_t left)
{
    Chunk<E> c;
    c.raw = u32x4{0, 0, 0, 0};
    if constexpr (VEC) {
        if (left > 0)
            c.raw = *reinterpret_cast<const u32x4 *>(p);
    } else if (left >= E::kChunk) {
        __builtin_memcpy(&c.raw, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < E::kChunk; ++i)
            if (i < left)
                c.e[i] = p[i];
    }
    return c.raw;
}

template <class E, bool VEC>
__device__ inline void store_chunk(typename E::T *p, const Chunk<E> &c, int64_t left)
{
    if constexpr (VEC) {
        if (left > 0)
            *reinterpret_cast<u32x4 *>(p) = c.raw;
    } else if (left >= E::kChunk) {
        __builtin_memcpy(p, &c.raw, 16);
    } else {
#pragma unroll
        for (int i = 0; i < E::kChunk; ++i)
            if (i < left)
                p[i] = c.e[i];
    }
}

// ---------------------------------------------------------------------------
// Wave-wide maximum
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xf, 0xf, false);
}

// The wave's largest x, in a scalar: rotations within rows of 16 lanes, then
// the four rows.  All lanes must be active.
__device__ inline uint32_t wave_max(uint32_t x)
{
    x = max(x, dpp<0x128>(x));   // row_ror:8
    x = max(x, dpp<0x124>(x));
    x = max(x, dpp<0x122>(x));
    x = max(x, dpp<0x121>(x));
    const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)x, 0), (uint32_t)__builtin_amdgcn_readlane((int)x, 16));
    const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)x, 32), (uint32_t)__builtin_amdgcn_readlane((int)x, 48));
    return max(a, b);
}

}  // namespace rows

#endif
