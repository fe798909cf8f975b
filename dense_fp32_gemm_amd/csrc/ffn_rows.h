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

// ---------------------------------------------------------------------------
// A row in 8 bits
// ---------------------------------------------------------------------------
// The definition is in binary64.  Its values are approximated in binary32 with a known
// relative error, and only those whose rounding that leaves open are computed in
// binary64: the elements that may be the row's largest, and those next to a
// rounding border (of 127 steps' binary32 error, one in ten thousand or fewer).  So the
// results are the definition's at a binary32 pass's cost.
//
//   approx(i, e, n)  the i-th chunk's element e (column n), to within ERROR
//   exact(n)         column n in binary64
//   unsure(i, e, n)  whether approx may be off by more
template <int TPR, int C, class E>
struct Int8Row {
    int N, j;
    bool there;                                      // the row
    int8_t *q;                                       // its start

    template <class Approx, class Exact, class Unsure>
    __device__ inline void write(RowSums<TPR> &over, float *scale, float error, Approx &&approx, Exact &&exact, Unsure &&unsure)
    {
        // NaN above infinity above every number, as whole numbers
        uint32_t top = 0;
        each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
#pragma unroll
            for (int e = 0; e < E::kChunk; ++e)
                if (n0 + e < N)
                    top = max(top, __float_as_uint(approx(i, e, n0 + e)) & 0x7fffffffu);
        });
        top = over.max32(top);
        // (rows up to 2^-120 get the smallest scale in any case)
        const float near = top > 0x7f800000u ? INFINITY : fmaxf(__uint_as_float(top) * (1.f - 4.f * error), 0x1p-120f);
        uint64_t most = 0;
        each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
            uint32_t check = 0;
#pragma unroll
            for (int e = 0; e < E::kChunk; ++e)
                if (n0 + e < N && (!(fabsf(approx(i, e, n0 + e)) < near) || unsure(i, e, n0 + e)))
                    check |= 1u << e;
#pragma unroll 1
            for (; check != 0; check &= check - 1) {
                const uint64_t y = __builtin_bit_cast(uint64_t, fabs(exact(n0 + (int)__builtin_ctz(check))));
                most = y > most ? y : most;
            }
        });
        most = over.max64(most);
        float s = fmaxf((float)(__builtin_bit_cast(double, most) / 127.0), 0x1p-126f);
        const bool bad = most >= 0x7ff0000000000000u || !(s < INFINITY);
        if (bad)
            s = __uint_as_float(0x7fc00000u);
        if (!there)
            return;
        if (j == 0)
            *scale = s;
        const float per = 1.f / s;
        // errors next to binary32's smallest numbers (of y, and of 1 / s) are not relative
        const bool edge = !(s > 0x1p-100f && s < 0x1p100f);
        each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
            struct {
                int8_t v[E::kChunk];
            } o;
            uint32_t check = 0;
#pragma unroll
            for (int e = 0; e < E::kChunk; ++e) {
                const float t = approx(i, e, n0 + e) * per, r = __builtin_rintf(t);
                if (!(fabsf(t - r) < 0.5f - fabsf(t) * (2.f * error)) || unsure(i, e, n0 + e) || (edge && t != 0.f))
                    check |= n0 + e < N ? 1u << e : 0u;
                o.v[e] = bad ? 0 : (int8_t)(int)fminf(fmaxf(r, -127.f), 127.f);
            }
            if (n0 + E::kChunk <= N) {
                __builtin_memcpy(q + n0, &o, sizeof o);
            } else {
#pragma unroll
                for (int e = 0; e < E::kChunk; ++e)
                    if (n0 + e < N)
                        q[n0 + e] = o.v[e];
            }
            if (bad)
                check = 0;
#pragma unroll 1
            for (; check != 0; check &= check - 1) {
                const int n = n0 + (int)__builtin_ctz(check);
                q[n] = (int8_t)(int)fmin(fmax(__builtin_rint(exact(n) / (double)s), -127.0), 127.0);
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
        call(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    else if (chunks <= 512)
        call(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    else if (chunks <= 1024)
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
    else if (chunks <= 2048)
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    else
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
}

}  // namespace ffn

#endif
