// Root-mean-square norm with the residual's addition, and its gradient (include/gemm_f32_ffn.h).
//
// A row belongs to TPR threads (a wave, or a workgroup), C chunks of 16 bytes each in
// registers: one pass over the data.  Rows that do not fit (C = 0) are read again
// where they are needed, chunk by chunk.  All kernels are bound by HBM.

#include "ffn_rows.h"

namespace ffn {
namespace {

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------
struct NormArgs {
    const void *X, *R;       // R: the residual, or NULL
    const float *weight;     // NULL: 1
    void *S;                 // NULL: not written
    void *Y;                 // of E, or 8 bits
    float *scale;            // 8 bits: of each row
    int64_t ldx, ldr, lds, ldy;
    double eps;
    int T, N;
};

// Bound by HBM: 8192 x 4096 fp16 with a residual, 268 MB, 43.2 us, 6.2 TB/s.  To 8 bits the rows' chains of steps show
// (sum, largest, factor, division): bf16, 235 MB, 50 us with warm caches, 56-57 from memory, 4.1-4.7 TB/s.
template <class E, bool VEC, bool INT8, int TPR, int C>
__global__ __launch_bounds__(kRowThreads<TPR>) void norm_kernel(NormArgs g)
{
    using T = typename E::T;
    constexpr int kRows = kRowsAtOnce<TPR>, K = E::kChunk;
    __shared__ typename RowJoin<TPR>::Pair slots[2][TPR / kWave];
    const int j = threadIdx.x % TPR;
    RowJoin<TPR> over{slots};
    auto weights = [&](float (&w)[K], int n0) {
        if (g.weight != nullptr)
            load_floats<E>(w, g.weight + n0, g.N - n0);
        else
#pragma unroll
            for (int e = 0; e < K; ++e)
                w[e] = 1.f;
    };
    float w[C > 0 ? C : 1][K];
    if constexpr (C > 0)
        each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) { weights(w[i], n0); });
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < g.T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + threadIdx.x / TPR;
        const bool there = t < g.T;
        const T *x = (const T *)g.X + (there ? t : 0) * g.ldx, *r = (const T *)g.R + (there && g.R != nullptr ? t : 0) * g.ldr;
        T *s = (T *)g.S + (there ? t : 0) * g.lds;
        // S as it is computed, before it is written over X or R
        auto summed = [&](Chunk<E> &z, int n0) {
            const int left = there ? g.N - n0 : 0;
            z.raw = load_chunk<E, VEC>(x + n0, left);
            if (g.R != nullptr) {
                Chunk<E> b;
                b.raw = load_chunk<E, VEC>(r + n0, left);
#pragma unroll
                for (int e = 0; e < K; ++e)
                    z.e[e] = (T)((float)z.e[e] + (float)b.e[e]);
            }
        };
        // ... and read again afterwards
        const bool kept = g.R != nullptr && g.S != nullptr;
        auto again = [&](Chunk<E> &z, int n0) {
            if (kept)
                z.raw = load_chunk<E, VEC>(s + n0, there ? g.N - n0 : 0);
            else
                summed(z, n0);
        };
        Chunk<E> z[C > 0 ? C : 1];
        double squares = 0.0;
        if constexpr (C > 0)                         // all loads, then their use
            each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) { summed(z[i], n0); });
        each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
            if constexpr (C == 0)
                summed(z[i], n0);
            if (kept && there)
                store_chunk<E, VEC>(s + n0, z[i], g.N - n0);
#pragma unroll
            for (int e = 0; e < K; ++e)
                squares = fma((double)(float)z[i].e[e], (double)(float)z[i].e[e], squares);
        });
        if constexpr (!INT8) {
            const float scale = (float)(1.0 / sqrt(over.sum(squares) / g.N + g.eps));
            each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
                if constexpr (C == 0) {
                    again(z[i], n0);
                    weights(w[i], n0);
                }
                Chunk<E> o;
#pragma unroll
                for (int e = 0; e < K; ++e)
                    o.e[e] = (T)((float)z[i].e[e] * scale * w[i][e]);
                if (there)
                    store_chunk<E, VEC>((T *)g.Y + t * g.ldy + n0, o, g.N - n0);
            });
        } else {
            int loaded = -1;                         // C = 0: the column whose chunk z and w hold
            auto open = [&](int i, int n0) {
                if constexpr (C == 0) {
                    if (loaded != n0) {
                        loaded = n0;
                        again(z[i], n0);
                        weights(w[i], n0);
                    }
                }
            };
            auto sure = [](int, int, int) { return false; };
            auto some = [&](int i, int e) { return (float)z[i].e[e] != 0.f; };
            // The largest S weight: a row's factor does not change which it is, so its approximation shares the
            // squares' exchange.
            auto product = [&](int i, int e, int n0) {
                open(i, n0);
                return (float)z[i].e[e] * w[i][e];
            };
            RowMost<TPR, C, E> most{g.N, j};
            uint64_t top = most.approximate(product);
            const double sum = over.sum_and_most(squares, top), scale = 1.0 / sqrt(sum / max(g.N, 1) + g.eps);
            const double largest = scale * most.exactly(over, top, 0x1p-23f, product,
                                                        [&](int i, int e, int) { return (double)pick(z[i], e) * (double)pick(w[i], e); },
                                                        sure, some);
            const float scale32 = (float)scale, most_product = __uint_as_float((uint32_t)top);
            if (there) {
                // S weight first: where the row's largest is an ordinary number, no product is infinite, and one under the normal
                // numbers is nothing beside a step.  (S r may be under them where a large weight makes it count.)
                Int8Row<TPR, C, E> row{g.N, j, (int8_t *)g.Y + t * g.ldy, false, !(most_product > 0x1p-99f && most_product < INFINITY)};
                row.write(largest, g.scale + t, [&](int i, int e, int n0) { return product(i, e, n0) * scale32; },
                          [&](int i, int e, int) { return (double)pick(z[i], e) * (double)pick(w[i], e) * scale; },
                          [](int, int) { return 0x1p-21f; }, sure, some);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient of the norm
// ---------------------------------------------------------------------------
struct NormGradArgs {
    const void *dY, *S, *dS;     // dS: NULL: none
    const float *weight;
    void *dX;                    // NULL: not computed
    float *partial;              // [workgroups][N] of dweight, NULL: not computed
    int64_t lddy, lds, ldds, lddx;
    double eps;
    int T, N;
};

// 16383 x 2048 bf16, 268 MB: 50.6 us, 5.3 TB/s (the norm above moves as much in 43.2: bound by the loads that eight
// waves a compute unit have in flight), and 5.4 us for the parts.
// A thread keeps its columns over all rows of its workgroup, and their part of dweight in
// registers; the workgroup's parts go to the workspace, which sum_kernel adds up.
// (C = 0: the parts are added in the workspace, by the thread whose columns they are.)
template <class E, bool VEC, int TPR, int C>
__global__ __launch_bounds__(kRowThreads<TPR>) void norm_grad_kernel(NormGradArgs g)
{
    using T = typename E::T;
    constexpr int kRows = kRowsAtOnce<TPR>, K = E::kChunk, kC = C > 0 ? C : 1;
    __shared__ typename RowJoin<TPR>::Pair slots[2][TPR / kWave];
    const int j = threadIdx.x % TPR;
    RowJoin<TPR> over{slots};
    float w[kC][K], sum[kC][K] = {};
    auto weights = [&](float (&v)[K], int n0) {
        if (g.weight != nullptr)
            load_floats<E>(v, g.weight + n0, g.N - n0);
        else
#pragma unroll
            for (int e = 0; e < K; ++e)
                v[e] = 1.f;
    };
    if constexpr (C > 0)
        each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) { weights(w[i], n0); });
    static_assert(C > 0 || kRows == 1, "a workgroup's part is added up in the workspace by one row's threads");
    float *mine = g.partial + (int64_t)blockIdx.x * g.N;
    bool first = true;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < g.T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + threadIdx.x / TPR;
        const bool there = t < g.T;
        const int64_t at = there ? t : 0;
        const T *dy = (const T *)g.dY + at * g.lddy, *s = (const T *)g.S + at * g.lds;
        const T *ds = (const T *)g.dS + (g.dS != nullptr ? at * g.ldds : 0);
        Chunk<E> d[kC], z[kC], more[kC];
        auto load = [&](int i, int n0) {
            const int left = there ? g.N - n0 : 0;
            d[i].raw = load_chunk<E, VEC>(dy + n0, left);
            z[i].raw = load_chunk<E, VEC>(s + n0, left);
        };
        if constexpr (C > 0)
            each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
                load(i, n0);
                more[i].raw = load_chunk<E, VEC>(ds + n0, there && g.dS != nullptr ? g.N - n0 : 0);
            });
        double squares = 0.0, along = 0.0;
        each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
            if constexpr (C == 0) {
                load(i, n0);
                weights(w[i], n0);
            }
#pragma unroll
            for (int e = 0; e < K; ++e) {
                const double v = (double)(float)z[i].e[e];
                squares = fma(v, v, squares);
                along = fma((double)((float)d[i].e[e] * w[i][e]), v, along);
            }
        });
        over.sums(squares, along);
        const double r = 1.0 / sqrt(squares / g.N + g.eps);
        const float r32 = (float)r, k = (float)(along / g.N * r * r);
        each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
            if constexpr (C == 0) {
                load(i, n0);
                weights(w[i], n0);
                more[i].raw = load_chunk<E, VEC>(ds + n0, there && g.dS != nullptr ? g.N - n0 : 0);
            }
            Chunk<E> o;
#pragma unroll
            for (int e = 0; e < K; ++e) {
                const float v = (float)z[i].e[e], u = (float)d[i].e[e];
                float x = r32 * fmaf(-v, k, u * w[i][e]);
                if (g.dS != nullptr)
                    x += (float)more[i].e[e];
                o.e[e] = (T)x;
                sum[i][e] = C == 0 ? u * (v * r32) : fmaf(u, v * r32, sum[i][e]);
            }
            if constexpr (C == 0) {
                if (g.partial != nullptr)
#pragma unroll
                    for (int e = 0; e < K; ++e)
                        if (n0 + e < g.N)
                            mine[n0 + e] = first ? sum[i][e] : mine[n0 + e] + sum[i][e];
            }
            if (there && g.dX != nullptr)
                store_chunk<E, VEC>((T *)g.dX + t * g.lddx + n0, o, g.N - n0);
        });
        first = false;
    }
    if constexpr (C > 0) {
        if (g.partial == nullptr)
            return;
        if constexpr (kRows > 1) {                   // the rows' parts, in order
            __shared__ float parts[kRows - 1][C * K][TPR];
            const int q = threadIdx.x / TPR;
#pragma unroll
            for (int i = 0; i < C * K; ++i)
                if (q > 0)
                    parts[q - 1][i][j] = sum[i / K][i % K];
            __syncthreads();
            if (q > 0)
                return;
#pragma unroll
            for (int r = 0; r < kRows - 1; ++r)
#pragma unroll
                for (int i = 0; i < C * K; ++i)
                    sum[i / K][i % K] += parts[r][i][j];
        }
        each_chunk<TPR, C, E>(g.N, j, [&](int i, int n0) {
#pragma unroll
            for (int e = 0; e < K; ++e)
                if (n0 + e < g.N)
                    mine[n0 + e] = sum[i][e];
        });
    }
}

// dweight[n] = sum of `parts` rows of partial: 16 columns a workgroup, 16 threads a column.
constexpr int kSumColumns = 16, kSumThreads = 256;
__global__ __launch_bounds__(kSumThreads) void sum_kernel(const float *partial, int parts, int N, float *dweight)
{
    constexpr int kRows = kSumThreads / kSumColumns;
    __shared__ double part[kRows][kSumColumns];
    const int c = threadIdx.x % kSumColumns, r = threadIdx.x / kSumColumns;
    for (int64_t n0 = (int64_t)blockIdx.x * kSumColumns; n0 < N; n0 += (int64_t)gridDim.x * kSumColumns) {
        double sum = 0.0;
        if (n0 + c < N) {
#pragma unroll 8
            for (int p = r; p < parts; p += kRows)
                sum += (double)partial[(int64_t)p * N + n0 + c];
        }
        part[r][c] = sum;
        __syncthreads();
        if (r == 0 && n0 + c < N) {
            double all = 0.0;
#pragma unroll
            for (int q = 0; q < kRows; ++q)
                all += part[q][c];
            dweight[n0 + c] = (float)all;
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(kSumThreads) void zero_kernel(float *p, int N)
{
    for (int64_t n = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; n < N; n += (int64_t)gridDim.x * kSumThreads)
        p[n] = 0.f;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Workgroups of the gradient at most, each with its part of dweight: on a whole MI355X four a compute unit up to 256
// threads a row (with 128 threads that is eight waves, half of what 256 have), two of 512, one of 1024
// (16384 x 512 fp16, four rows a workgroup, whose parts are joined in LDS: 18.5 us; 24.5 with a part in the workspace
// for each, which allows a quarter of the workgroups).
constexpr int kGradParts = 1024;
int grad_parts(int T) { return T < kGradParts ? T : kGradParts; }
int grad_grid(int T, int rows, int threads)
{
    const int64_t need = ceil_div(T, rows), fit = gemm_f32_internal::current_device().cus * 4 * 256 / threads;
    const int64_t most = fit < kGradParts ? fit : kGradParts;
    return (int)(need < most ? need : most);
}

bool bad_eps(float eps) { return !(eps > 0.f && eps < INFINITY); }

int norm_call(int type, int T, int N, const void *X, int ldx, const void *R, int ldr, const float *weight, float eps,
              void *S, int lds, void *Y, int ldy, float *scale, bool int8, hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (bad_size(T) || bad_size(N))
        return GEMM_F32_ERR_DIM;
    if (short_ld(ldx, N) || (R != nullptr && short_ld(ldr, N)) || (R != nullptr && S != nullptr && short_ld(lds, N)) || short_ld(ldy, N))
        return GEMM_F32_ERR_LD;
    if (bad_eps(eps))
        return GEMM_F32_ERR_OPTION;
    if (T == 0 || (N == 0 && !int8))
        return GEMM_F32_OK;
    if ((N > 0 && (X == nullptr || Y == nullptr)) || (int8 && scale == nullptr))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(X, b) || !aligned_to(R, b) || !aligned_to(weight, 4) || !aligned_to(S, b) || (!int8 && !aligned_to(Y, b)) ||
        !aligned_to(scale, 4))
        return GEMM_F32_ERR_ALIGN;
    const NormArgs g{X, R, weight, S, Y, scale, ldx, ldr, lds, ldy, (double)eps, T, N};
    const bool vec = chunk_rows(type, X, ldx, N) && (R == nullptr || chunk_rows(type, R, ldr, N)) &&
                     (R == nullptr || S == nullptr || chunk_rows(type, S, lds, N)) && (int8 || chunk_rows(type, Y, ldy, N));
    with_type(type, [&](auto e) {
        using E = decltype(e);
        with_row<E>(N, [&](auto tpr, auto c) {
            constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value, NT = kRowThreads<TPR>;
            const int grid = row_grid(T, kRowsAtOnce<TPR>, NT);
            auto launch = [&](auto v, auto q) {
                norm_kernel<E, decltype(v)::value, decltype(q)::value, TPR, C><<<grid, NT, 0, stream>>>(g);
            };
            if (vec)
                int8 ? launch(std::true_type{}, std::true_type{}) : launch(std::true_type{}, std::false_type{});
            else
                int8 ? launch(std::false_type{}, std::true_type{}) : launch(std::false_type{}, std::false_type{});
        });
    });
    return launched();
}

}  // namespace
}  // namespace ffn

using namespace ffn;

extern "C" {

int gemm_f32_rms_norm(int type, int T, int N, const void *X, int ldx, const void *residual, int ldr, const float *weight,
                      float eps, void *sum, int lds, void *Y, int ldy, hipStream_t stream)
{
    return norm_call(type, T, N, X, ldx, residual, ldr, weight, eps, sum, lds, Y, ldy, nullptr, false, stream);
}

int gemm_f32_rms_norm_int8(int type, int T, int N, const void *X, int ldx, const void *residual, int ldr,
                           const float *weight, float eps, void *sum, int lds, int8_t *Q, int ldq, float *scale,
                           hipStream_t stream)
{
    return norm_call(type, T, N, X, ldx, residual, ldr, weight, eps, sum, lds, Q, ldq, scale, true, stream);
}

size_t gemm_f32_rms_norm_grad_ws_size(int T, int N)
{
    if (T <= 0 || N <= 0 || bad_size(T) || bad_size(N))
        return 0;
    return (size_t)ceil_div((int64_t)grad_parts(T) * N * 4, 16) * 16;
}

int gemm_f32_rms_norm_grad(int type, int T, int N, const void *dY, int lddy, const void *S, int lds, const float *weight,
                           float eps, const void *dsum, int ldds, void *dX, int lddx, float *dweight, void *workspace,
                           size_t workspace_bytes, hipStream_t stream)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (bad_size(T) || bad_size(N))
        return GEMM_F32_ERR_DIM;
    if (short_ld(lddy, N) || short_ld(lds, N) || (dsum != nullptr && short_ld(ldds, N)) || (dX != nullptr && short_ld(lddx, N)))
        return GEMM_F32_ERR_LD;
    if (bad_eps(eps))
        return GEMM_F32_ERR_OPTION;
    if (N == 0 || (dX == nullptr && dweight == nullptr) || (T == 0 && dweight == nullptr))
        return GEMM_F32_OK;
    if (T > 0 && (dY == nullptr || S == nullptr))
        return GEMM_F32_ERR_NULL;
    const int b = type_bytes(type);
    if (!aligned_to(dY, b) || !aligned_to(S, b) || !aligned_to(weight, 4) || !aligned_to(dsum, b) || !aligned_to(dX, b) ||
        !aligned_to(dweight, 4))
        return GEMM_F32_ERR_ALIGN;
    if (T > 0 && dweight != nullptr &&
        (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < gemm_f32_rms_norm_grad_ws_size(T, N)))
        return GEMM_F32_ERR_WORKSPACE;
    const int sum_grid = (int)(ceil_div(N, kSumColumns) < 65536 ? ceil_div(N, kSumColumns) : 65536);
    if (T == 0) {
        zero_kernel<<<sum_grid, kSumThreads, 0, stream>>>(dweight, N);
        return launched();
    }
    float *partial = dweight != nullptr ? (float *)workspace : nullptr;
    const NormGradArgs g{dY, S, dsum, weight, dX, partial, lddy, lds, ldds, lddx, (double)eps, T, N};
    const bool vec = chunk_rows(type, dY, lddy, N) && chunk_rows(type, S, lds, N) && (dsum == nullptr || chunk_rows(type, dsum, ldds, N)) &&
                     (dX == nullptr || chunk_rows(type, dX, lddx, N));
    int parts = 0;
    with_type(type, [&](auto e) {
        using E = decltype(e);
        with_row<E>(N, [&](auto tpr, auto c) {
            constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value, NT = kRowThreads<TPR>;
            const int grid = grad_grid(T, kRowsAtOnce<TPR>, NT);
            parts = grid;
            if (vec)
                norm_grad_kernel<E, true, TPR, C><<<grid, NT, 0, stream>>>(g);
            else
                norm_grad_kernel<E, false, TPR, C><<<grid, NT, 0, stream>>>(g);
        });
    });
    const int rc = launched();
    if (rc != GEMM_F32_OK || dweight == nullptr)
        return rc;
    sum_kernel<<<sum_grid, kSumThreads, 0, stream>>>(partial, parts, N, dweight);
    return launched();
}

}  // extern "C"
