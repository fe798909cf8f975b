// Rows in 8 bits, as they are or gated (include/gemm_f32_ffn.h).  A row belongs to the
// threads of a wave or a workgroup, in registers (see ffn_rows.h).  Bound by HBM.

#include "ffn_rows.h"

namespace ffn {
namespace {

struct QuantizeArgs {
    const void *X;
    int8_t *Q;
    float *scale;
    int64_t ldx, ldq;
    int T, N;
};

// From where on to the left a gate's sigmoid is no normal binary32 number (as a factor of y it may
// still count).
template <int GATE>
constexpr float gate_left()
{
    return GATE == GEMM_F32_GATE_SILU ? -80.f : GATE == GEMM_F32_GATE_GELU ? -12.f : -9.5f;
}

// 8192 x 4096 as they are, bf16, 101 MB: 23 us, 4.4 TB/s.  silu, 4096 x 8192 fp16, 168 MB: 44 us with warm caches, 52
// from memory, 3.2-3.8 TB/s: a wave's chain (gates, the row's largest in binary64, division, borders) with 16 waves
// a compute unit; gelu_tanh 49.  gelu 87: as many elements go through binary64 (gate_error() is the same), but erfc()
// there costs several times an exponential, once a row at least and behind a barrier, the binary32 polynomial is longer,
// and of 1024 threads a row the variants spill (25 registers in bf16, 14 in half).
// 16-bit types: registers for three waves a SIMD, which gelu's two chunks otherwise just miss in some variants (169 of
// 168; 8192 x 4096 bf16 with one too many: 79 us, 64 without).  binary32 fits four by itself.
template <class E, bool VEC, int GATE, int TPR, int C>
__global__ __launch_bounds__(kRowThreads<TPR>, E::kBytes == 2 && TPR < 1024 ? 3 : 1) void quantize_kernel(QuantizeArgs g)
{
    using T = typename E::T;
    constexpr int kRows = kRowsAtOnce<TPR>, K = E::kChunk, kC = C > 0 ? C : 1;
    constexpr bool kGated = GATE != GEMM_F32_GATE_NONE, kSmallGates = !std::is_same<E, F16>::value;   // half has none under kSmall
    // How a gate far on the left is found: compared one by one where 1024 threads of bfloat16 have the chunks (14336 and
    // 16384 columns, 4096 rows: silu 105 and 108 us, gelu 163 and 172; by the smallest of the thread's 107 and 110, 172 and
    // 179), else by the smallest (8192 x 4096 bf16: silu 41, compared 46; 4096 x 6000 binary32: gelu 79, compared 84).
    constexpr bool kCompare = std::is_same<E, Bf16>::value && TPR == 1024 && C > 0;
    __shared__ typename RowJoin<TPR>::Pair slots[2][TPR / kWave];
    const int j = threadIdx.x % TPR;
    RowJoin<TPR> over{slots};
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < g.T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + threadIdx.x / TPR;
        const bool there = t < g.T;
        const T *x = (const T *)g.X + (there ? t : 0) * g.ldx;
        Chunk<E> a[kC], b[kGated ? kC : 1];
        float y[kC][kGated ? K : 1];
        auto load = [&](int i, int n0) {
            const int left = there ? g.N - n0 : 0;
            a[i].raw = load_chunk<E, VEC>(x + n0, left);
            if constexpr (kGated)
                b[i].raw = load_chunk<E, VEC>(x + g.N + n0, left);
        };
        bool far = false;
        float lowest = 0.f, heavy = 0.f;             // the smallest gate, the largest of what they gate
        auto open = [&](int i) {                     // the chunk's values
            if constexpr (kGated)
#pragma unroll
                for (int e = 0; e < K; e += 2) {
                    const float p = (float)a[i].e[e], q = (float)a[i].e[e + 1], u = (float)b[i].e[e], v = (float)b[i].e[e + 1];
                    y[i][e] = gate<GATE>(p) * u;
                    y[i][e + 1] = gate<GATE>(q) * v;
                    if (kCompare)
                        far |= p < gate_left<GATE>() || q < gate_left<GATE>();
                    else
                        lowest = min3(lowest, p, q);
                    if (kSmallGates)
                        heavy = max3(heavy, fabsf(u), fabsf(v));
                }
        };
        if constexpr (C > 0) {
            each_chunk<TPR, C, E>(g.N, j, load);
            each_chunk<TPR, C, E>(g.N, j, [&](int i, int) { open(i); });
        }
        int loaded = -1;                             // C = 0: the column whose chunk a, b and y hold
        auto approx = [&](int i, int e, int n0) {
            if constexpr (C == 0) {
                if (loaded != n0) {
                    loaded = n0;
                    load(i, loaded);
                    open(i);
                }
            }
            if constexpr (kGated)
                return y[i][e];
            else
                return (float)a[i].e[e];
        };
        auto exact = [&](int i, int e, int) {
            if constexpr (kGated)
                return gate64<GATE>((double)pick(a[i], e)) * (double)pick(b[i], e);
            else
                return (double)pick(a[i], e);
        };
        auto unsure = [&](int i, int e, int) { return kGated && (float)a[i].e[e] < gate_left<GATE>(); };
        auto some = [&](int i, int e) { return (float)a[i].e[e] != 0.f; };
        RowMost<TPR, C, E> most{g.N, j};
        uint64_t top = most.approximate(approx);
        if constexpr (kGated && kSmallGates) {
            // (the row's largest is that of a wave at least)
            bool small = false;
            if (__ballot(heavy * kHeavy > __uint_as_float((uint32_t)top)) != 0) {
                each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
#pragma unroll
                    for (int e = 0; e < K; ++e) {
                        approx(i, e, n0);
                        const float x = fabsf((float)a[i].e[e]);         // act(x) is about x / 2
                        small |= x != 0.f && x < kSmall;
                    }
                });
                if (__ballot(small) != 0)
                    top |= 1ull << 32;               // above every magnitude; exactly() then needs none
            }
        }
        over.most(top);
        most.every = top >> 32 != 0;
        double largest = (double)__uint_as_float((uint32_t)top);
        most.loose = kGated && (kCompare ? far : lowest < gate_left<GATE>());
        if constexpr (kGated)
            largest = most.exactly(over, top, kGateFar, approx, exact, unsure, some);
        if (there) {
            Int8Row<TPR, C, E> row{g.N, j, g.Q + t * g.ldq, most.loose, most.every};
            row.write(largest, g.scale + t, approx, exact,
                      [&](int i, int e) { return kGated ? gate_error<GATE>((float)a[i].e[e]) : 0x1p-23f; }, unsure, some);
        }
    }
}

}  // namespace
}  // namespace ffn

using namespace ffn;

extern "C" {

int gemm_f32_quantize(int type, int gate, int T, int N, const void *X, int ldx, int8_t *Q, int ldq, float *scale,
                      hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (bad_size(T) || bad_size(N) || (gate != GEMM_F32_GATE_NONE && N > kMaxSize / 2))
        return GEMM_F32_ERR_DIM;
    if (short_ld(ldx, gate != GEMM_F32_GATE_NONE ? 2 * N : N) || short_ld(ldq, N))
        return GEMM_F32_ERR_LD;
    if (gate != GEMM_F32_GATE_NONE && !known_gate(gate))
        return GEMM_F32_ERR_OPTION;
    if (T == 0)
        return GEMM_F32_OK;
    if ((N > 0 && (X == nullptr || Q == nullptr)) || scale == nullptr)
        return GEMM_F32_ERR_NULL;
    if (!aligned_to(X, type_bytes(type)) || !aligned_to(scale, 4))
        return GEMM_F32_ERR_ALIGN;
    const QuantizeArgs g{X, Q, scale, ldx, ldq, T, N};
    const bool vec = chunk_rows(type, X, ldx, N);
    with_type(type, [&](auto e) {
        using E = decltype(e);
        with_gate(gate, [&](auto kind) {
            with_row<E>(N, [&](auto tpr, auto c) {
                constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value, NT = kRowThreads<TPR>;
                const int grid = row_grid(T, kRowsAtOnce<TPR>, NT);
                if (vec)
                    quantize_kernel<E, true, decltype(kind)::value, TPR, C><<<grid, NT, 0, stream>>>(g);
                else
                    quantize_kernel<E, false, decltype(kind)::value, TPR, C><<<grid, NT, 0, stream>>>(g);
            });
        });
    });
    return launched();
}

}  // extern "C"
