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

// Rotations within rows of 16 lanes, then the four rows' first lanes, in scalars.
template <int CTRL>
__device__ inline uint64_t dpp64(uint64_t x)
{
    return (uint64_t)dpp<CTRL>((uint32_t)(x >> 32)) << 32 | dpp<CTRL>((uint32_t)x);
}
__device__ inline uint64_t lane64(uint64_t x, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}
template <class Join>
__device__ inline uint64_t wave_join(uint64_t v, Join &&join)
{
    v = join(v, dpp64<0x128>(v));   // row_ror:8
    v = join(v, dpp64<0x124>(v));
    v = join(v, dpp64<0x122>(v));
    v = join(v, dpp64<0x121>(v));
    return join(join(lane64(v, 0), lane64(v, 16)), join(lane64(v, 32), lane64(v, 48)));
}
__device__ inline uint64_t add64(uint64_t a, uint64_t b)
{
    return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b));
}
__device__ inline uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Reductions over a row's threads, the same in each: of a sum in binary64 and of something else,
// with one barrier.  Two slots in turn: a slot is written again after the barrier that its readers pass next.
template <int TPR>
struct RowJoin {
    static constexpr int kWaves = TPR / kWave;
    struct Pair {
        uint64_t a, b;
    };
    Pair (*slots)[kWaves];                           // LDS [2][kWaves]
    int at = 0;

    // a and b are the same in a wave
    template <class JoinA, class JoinB>
    __device__ inline void join(uint64_t &a, uint64_t &b, JoinA &&join_a, JoinB &&join_b)
    {
        if constexpr (kWaves > 1) {
            at ^= 1;
            if (threadIdx.x % kWave == 0)
                slots[at][threadIdx.x / kWave] = Pair{a, b};
            __syncthreads();
            a = slots[at][0].a, b = slots[at][0].b;
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                a = join_a(a, slots[at][w].a);
                b = join_b(b, slots[at][w].b);
            }
        }
    }
    __device__ inline void sums(double &x, double &y)
    {
        uint64_t a = wave_join(__builtin_bit_cast(uint64_t, x), add64), b = wave_join(__builtin_bit_cast(uint64_t, y), add64);
        join(a, b, add64, add64);
        x = __builtin_bit_cast(double, a), y = __builtin_bit_cast(double, b);
    }
    __device__ inline double sum(double x)
    {
        uint64_t a = wave_join(__builtin_bit_cast(uint64_t, x), add64), b = 0;
        join(a, b, add64, add64);
        return __builtin_bit_cast(double, a);
    }
    // the row's largest b beside; b is the same in a wave
    __device__ inline double sum_and_most(double x, uint64_t &b)
    {
        uint64_t a = wave_join(__builtin_bit_cast(uint64_t, x), add64);
        join(a, b, add64, max64);
        return __builtin_bit_cast(double, a);
    }
    __device__ inline void most(uint64_t &b)
    {
        uint64_t a = 0;
        join(a, b, add64, max64);
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
__host__ __device__ inline void each_chunk(int N, int j, Fn &&f)
{
    if constexpr (C > 0) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            f(i, (i * TPR + j) * E::kChunk);
    } else {
        // unsigned: the last step goes past a row by up to 8192, more than sizes leave under 2^31
        static_assert((uint32_t)kMaxSize + TPR * E::kChunk > (uint32_t)kMaxSize, "the last step stays in 32 bits");
        for (uint32_t n = j * E::kChunk; n < (uint32_t)N; n += TPR * E::kChunk)
            f(0, (int)n);
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
// results are the definition's at a binary32 pass's cost.
//
//   approx(i, e, n0)  the i-th chunk's element e (column n0 + e); 0 past the row's end
//   error(i, e)       how far that may be off, relative, at most most_error
//   exact(i, e, n0)   the same in binary64; e is no constant (see pick())
//   unsure(i, e, n0)  whether approx may be off by more; asked where `loose` says that one of the thread's may be
//   some(i, e)        whether exact() may be other than 0
//
// A factor of approx under binary32's normal numbers is off by up to 2^-150 instead, and the value by that times the
// other factor.  In steps of the scale, 2^-7 of the row's largest, that is under 2^-25, beside errors of twice
// error() (a value is looked at from half a step on), unless the other factor is beyond 2^118 of the row's largest.
// There `every` element that may be other than 0 is computed in binary64.
constexpr float kHeavy = 0x1p-118f, kSmall = 0x1p-120f;
// The largest and the smallest of three numbers in one instruction (fmaxf() first quiets NaN); NaN if one is.
__device__ inline float max3(float a, float b, float c) { return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c); }
__device__ inline float min3(float a, float b, float c) { return __builtin_elementwise_minimum(__builtin_elementwise_minimum(a, b), c); }

// Which of a chunk's first `left` elements are so.
template <class E, class Is>
__device__ inline uint32_t ones(int left, Is &&is)
{
    uint32_t all = 0;
#pragma unroll
    for (int e = 0; e < E::kChunk; ++e)
        if (e < left && is(e))
            all |= 1u << e;
    return all;
}

// A row's largest magnitude in two steps, as whole numbers (NaN above infinity above every number):
// that of approx() among the thread's elements, of which the caller makes the row's, and from
// that the largest of exact().
template <int TPR, int C, class E>
struct RowMost {
    int N, j;
    uint32_t mine = 0;
    bool loose = false;                              // whether any of the thread's elements is unsure
    bool every = false;                              // the same in all of the row's threads

    // The wave's.
    template <class Approx>
    __device__ inline uint64_t approximate(Approx &&approx)
    {
        each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
#pragma unroll
            for (int e = 0; e < E::kChunk; ++e)
                mine = max(mine, __float_as_uint(approx(i, e, n0)) & 0x7fffffffu);
        });
        return wave_max(mine);
    }
    // The row's.
    template <class Approx, class Exact, class Unsure, class Some>
    __device__ inline double exactly(RowJoin<TPR> &over, uint64_t row_top, float most_error, Approx &&approx, Exact &&exact, Unsure &&unsure,
                                     Some &&some) const
    {
        // Below `near` nothing is the largest.  Next to binary32's smallest numbers errors are not relative.
        const uint32_t top = (uint32_t)row_top;
        const float near = top > 0x7f800000u ? INFINITY : __uint_as_float(top) * (1.f - 4.f * most_error);
        const bool small = near < 0x1p-100f || every;
        uint64_t most = 0;
        if (!(__uint_as_float(mine) < near) || loose || small)
            each_chunk<TPR, C, E>(N, j, [&](int i, int n0) {
                uint32_t check = 0;
#pragma unroll
                for (int e = 0; e < E::kChunk; ++e) {
                    const bool large = !(fabsf(approx(i, e, n0)) < near);
                    if (n0 + e < N && (small ? some(i, e) : large))
                        check |= 1u << e;
                }
                if (loose)                           // few waves have any
                    check |= ones<E>(N - n0, [&](int e) { return unsure(i, e, n0); });
#pragma unroll 1
                for (; check != 0; check &= check - 1)
                    most = max64(most, __builtin_bit_cast(uint64_t, fabs(exact(i, (int)__builtin_ctz(check), n0))));
            });
        if (__ballot(most != 0) != 0)                // few waves have any
            most = wave_join(most, max64);
        over.most(most);
        return __builtin_bit_cast(double, most);
    }
};

// A row's scale from the largest magnitude of its exact values, and its 8-bit numbers.
template <int TPR, int C, class E>
struct Int8Row {
    int N, j;
    int8_t *q;                                       // the row's start
    bool loose, every;                               // as RowMost's (every: of this thread)

    template <class Approx, class Exact, class Error, class Unsure, class Some>
    __device__ inline void write(double most, float *scale, Approx &&approx, Exact &&exact, Error &&error, Unsure &&unsure, Some &&some)
    {
        constexpr int K = E::kChunk;
        float s = fmaxf((float)(most / 127.0), 0x1p-126f);
        const bool bad = !(most < INFINITY) || !(s < INFINITY);
        if (bad)
            s = __uint_as_float(0x7fc00000u);
        if (j == 0)
            *scale = s;
        const float per = 1.f / s;
        // Next to binary32's ends (of y, of s and of 1 / s) errors are not relative.
        const bool edge = !(s > 0x1p-100f && s < 0x1p100f) || every;
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
                    if (n0 + e < N && (!(fmaf(fabsf(t), 2.f * error(i, e), fabsf(t - __builtin_rintf(t))) < 0.5f) || (edge && some(i, e))))
                        check |= 1u << e;
                }
                if (loose)
                    check |= ones<E>(N - n0, [&](int e) { return unsure(i, e, n0); });
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
// there are.  Two chunks a thread where a wave alone would hold more (us, 8192 rows of 2048, bf16: to 8 bits through the
// norm 26.9 with 128 x 2, 30.9 with 256 x 1; of 8192: the gradient 92 with 512 x 2, 103 with 256 x 4, to 8 bits
// through the norm 110 and 150, as they are 45 and 39; of 16384: through the norm 123 with 1024 x 2, 140 with 512 x 4).
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
        call(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    else if (chunks <= 2048)
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    else
        call(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
}

}  // namespace ffn

#endif
