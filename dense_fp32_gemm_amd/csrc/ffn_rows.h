// Rows over the threads of a wave or a workgroup: loops, reductions, a row in 8 bits, and
// which rows get how many threads.
#ifndef GEMM_F32_FFN_ROWS_H
#define GEMM_F32_FFN_ROWS_H

#include <type_traits>

#include "ffn_gate.h"

namespace ffn {

// ---------------------------------------------------------------------------
// A row's threads
// ---------------------------------------------------------------------------
// Threads a workgroup has, and rows it works on side by side.
template <int TPR>
constexpr int kRowsAtOnce = TPR == kWave ? 4 : 1;
template <int TPR>
constexpr int kRowThreads = TPR * kRowsAtOnce<TPR>;

__device__ inline double wave_sum(double v)
{
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2)
        v += __shfl_xor(v, d);
    return v;
}

__device__ inline uint64_t wave_max64(uint64_t v)
{
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}

// Reductions over a row's threads, the same in each.  Two slots in turn: a slot is
// written again after the barrier that its readers pass next.
template <int TPR>
struct RowSums {
    static constexpr int kWaves = TPR / kWave;
    uint64_t (*slots)[kWaves];                       // LDS [2][kWaves]
    int at = 0;

    __device__ inline const uint64_t *exchange(uint64_t mine)
    {
        at ^= 1;
        if (threadIdx.x % kWave == 0)
            slots[at][threadIdx.x / kWave] = mine;
        __syncthreads();
        return slots[at];
    }
    __device__ inline double sum(double v)
    {
        v = wave_sum(v);
        if constexpr (kWaves > 1) {
            const uint64_t *all = exchange(__builtin_bit_cast(uint64_t, v));
            v = 0.0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                v += __builtin_bit_cast(double, all[w]);
        }
        return v;
    }
    __device__ inline uint32_t max32(uint32_t v)
    {
        v = wave_max(v);
        if constexpr (kWaves > 1) {
            const uint64_t *all = exchange(v);
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                v = max(v, (uint32_t)all[w]);
        }
        return v;
    }
    __device__ inline uint64_t max64(uint64_t v)
    {
        v = wave_max64(v);
        if constexpr (kWaves > 1) {
            const uint64_t *all = exchange(v);
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                v = all[w] > v ? all[w] : v;
        }
        return v;
    }
};

template <class E>
__device__ inline void load_floats(float (&w)[E::kChunk], const float *p, int left)
{
    if (left >= E::kChunk) {
        __builtin_memcpy(w, p, sizeof w);
    } else {
#pragma unroll
        for (int e = 0; e < E::kChunk; ++e)
            w[e] = e < left ? p[e] : 0.f;
    }
}

// Chunks of a row: f(i, column) for each of this thread's, C of them in registers (the
// index is a constant) or as many as the row has.
template <int TPR, int C, class E, class Fn>
__device__ inline void each_chunk(int N, int j, Fn &&f)
{
    if constexpr (C > 0) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            f(i, (i * TPR + j) * E::kChunk);
    } else {
        for (int n = j * E::kChunk; n < N; n += TPR * E::kChunk)
            f(0, n);
    }
}

// Element e of 16 bytes, or of K floats, in registers, where e is no constant.  (Whole vectors, then
// selections: selections between elements of an array become loads from one in memory.)
__device__ inline uint32_t pick(u32x4 v, int e) { return e < 2 ? (e == 0 ? v[0] : v[1]) : e == 2 ? v[2] : v[3]; }
template <class E>
__device__ inline float pick(const Chunk<E> &c, int e)
{
    if constexpr (E::kBytes == 4)
        return __uint_as_float(pick(c.raw, e));
    else
        return (float)__builtin_bit_cast(typename E::T, (uint16_t)(pick(c.raw, e / 2) >> (e % 2 * 16)));
}
template <int K>
__device__ inline float pick(const float (&c)[K], int e)
{
    u32x4 v[K / 4];
    __builtin_memcpy(v, c, sizeof v);
    const uint32_t low = pick(v[0], e % 4), high = pick(v[K / 4 - 1], e % 4);
    return __uint_as_float(e < 4 ? low : high);
}

// ---------------------------------------------------------------------------
// A row in 8 bits
// ---------------------------------------------------------------------------
// The definition is in binary64.  Its values are approximated in binary32 with a known
// relative error, and only those whose rounding that leaves open are computed in
// binary64: the elements that may be the row's largest, and those next to a
// rounding border (of 127 steps' binary32 error, one in ten thousand or fewer).  So the
// results are the definition's at a binary32 pass's cost.  SURE: approx is exact.
//
//   approx(i, e, n0)  the i-th chunk's element e (column n0 + e); 0 past the row's end
//   error(i, e)       how far that may be off, relative, at most most_error
//   exact(i, e, n0)   the same in binary64; e is no constant (see pick())
//   unsure(i, e, n0)  whether approx may be off by more
template <int TPR, int C, class E, bool SURE>
struct Int8Row {
    int N, j;
    bool there;                                      // the row
    int8_t *q;                                       // its start

    template <class Approx, class Exact, class Error, class Unsure>
    __device__ inline void write(RowSums<TPR> &over, float *scale, float most_error, Approx &&approx, Exact &&exact, Error &&error,
                                 Unsure &&unsure)
    {
        constexpr int K = E::kChunk;
        constexpr uint32_t kInf = 0x7f800000u;
        // NaN above infinity above every number, as whole numbers
        uint32_t mine = 0;
        bool loose = false;
        each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
#pragma unroll
            for (int e = 0; e < K; ++e) {
                mine = max(mine, __float_as_uint(approx(i, e, n0)) & 0x7fffffffu);
                loose |= unsure(i, e, n0);
            }
        });
        const uint32_t top = over.max32(mine);
        uint64_t most = 0;
        if constexpr (SURE) {
            most = __builtin_bit_cast(uint64_t, (double)__uint_as_float(top));
        } else {
            // Below `near` nothing is the row's largest.  (Rows up to 2^-120 get the smallest scale in any case.)
            const float near = top > kInf ? INFINITY : fmaxf(__uint_as_float(top) * (1.f - 4.f * most_error), 0x1p-120f);
            if (!(__uint_as_float(mine) < near) || loose)
                each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
                    uint32_t check = 0;
#pragma unroll
                    for (int e = 0; e < K; ++e)
                        if (n0 + e < N && (!(fabsf(approx(i, e, n0)) < near) || unsure(i, e, n0)))
                            check |= 1u << e;
#pragma unroll 1
                    for (; check != 0; check &= check - 1) {
                        const uint64_t y = __builtin_bit_cast(uint64_t, fabs(exact(i, (int)__builtin_ctz(check), n0)));
                        most = y > most ? y : most;
                    }
                });
            most = over.max64(most);
        }
        float s = fmaxf((float)(__builtin_bit_cast(double, most) / 127.0), 0x1p-126f);
        const bool bad = most >= 0x7ff0000000000000u || !(s < INFINITY);
        if (bad)
            s = __uint_as_float(0x7fc00000u);
        if (!there)
            return;
        if (j == 0)
            *scale = s;
        const float per = 1.f / s;
        // Next to binary32's ends (of y, of s and of 1 / s) errors are not relative.
        const bool edge = top >= kInf || !(s > 0x1p-100f && s < 0x1p100f);
        constexpr float kMagic = 0x1.8p23f;          // t + kMagic has t's nearest whole number in its low bits
        each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
            float worst = 0.f;
            union {
                uint32_t word[K / 4];
                int8_t v[K];
            } o;
#pragma unroll
            for (int e = 0; e < K; e += 4) {
                uint32_t b[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float t = approx(i, e + u, n0) * per, r = t + kMagic;
                    worst = fmaxf(worst, fmaf(fabsf(t), 2.f * error(i, e + u), fabsf(t - (r - kMagic))));
                    b[u] = __float_as_uint(r);
                }
                const uint32_t low = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), high = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
                o.word[e / 4] = bad ? 0u : __builtin_amdgcn_perm(high, low, 0x05040100u);
            }
            if (n0 + K <= N) {
                __builtin_memcpy(q + n0, &o, sizeof o);
            } else {
#pragma unroll
                for (int e = 0; e < K; ++e)
                    if (n0 + e < N)
                        q[n0 + e] = o.v[e];
            }
            if (!bad && (worst >= 0.5f || loose || edge)) {
                uint32_t check = 0;
#pragma unroll
                for (int e = 0; e < K; ++e) {
                    const float t = approx(i, e, n0) * per;
                    if (n0 + e < N && (!(fmaf(fabsf(t), 2.f * error(i, e), fabsf(t - __builtin_rintf(t))) < 0.5f) || unsure(i, e, n0) ||
                                       (edge && t != 0.f)))
                        check |= 1u << e;
                }
#pragma unroll 1
                for (; check != 0; check &= check - 1) {
                    const int e = (int)__builtin_ctz(check);
                    q[n0 + e] = (int8_t)(int)fmin(fmax(__builtin_rint(exact(i, e, n0) / (double)s), -127.0), 127.0);
                }
            }
        });
    }
};

// Workgroups that run side by side on the device, more or less: rows beyond them go to the same
// workgroups, which hold weights and sums over rows.
constexpr int kRowWorkgroups = 8;                    // of a compute unit, 256 threads each
inline int row_grid(int T, int rows, int threads)
{
    const int64_t need = ceil_div(T, rows), most = gemm_f32_internal::current_device().cus * kRowWorkgroups * 256 / threads;
    return (int)(need < most ? need : most);
}

// Calls f(threads per row, chunks per thread) for rows of N elements; 0 chunks: as many as
// there are.
template <class E, class Fn>
void with_row(int N, Fn &&f)
{
    const int64_t chunks = ceil_div(N, E::kChunk);
    auto call = [&](auto tpr, auto c) { f(tpr, c); };
    if (chunks <= 64)
        call(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (chunks <= 128)
        call(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    else if (chunks <= 256)
        call(std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{});
    else if (chunks <= 512)
        call(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    else if (chunks <= 1024)
        call(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    else if (chunks <= 2048)
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    else
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
}

}  // namespace ffn

#endif
