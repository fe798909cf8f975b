// Routing of tokens to experts, its gradient, and the slot map
// (include/gemm_f32_rows.h).
//
//  * route_kernel: one wave per token.  A lane holds every 64th expert; the
//    choice is k rounds of a wave-wide maximum over 64-bit keys.
//  * route_grad_kernel: one wave per token, the same layout.
//  * count_slots, place_slots: a stable counting sort of the slots by expert,
//    a workgroup per kSlotChunk slots.
//
// Scores are binary64: which expert is taken hangs on differences between
// neighbouring scores, and a score rounded to 24 bits makes ties (and with
// them wrong choices) of what the formula tells apart.

#include "rows_common.h"

namespace rows {
namespace {

constexpr int kRouteWaves = 4;       // tokens of a workgroup
constexpr int kRouteThreads = kRouteWaves * kWave;

struct RouteArgs {
    const void *logits;
    const float *bias;
    float *weight;
    int *index;
    int64_t ldl;
    int T, E, k, groups, keep_groups, group_top;
    bool softmax, normalize;
    float scale;
};

// ---------------------------------------------------------------------------
// Wave-wide sums
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ inline double dpp_double(double x)
{
    const uint64_t u = __double_as_longlong(x);
    const uint32_t lo = dpp<CTRL>((uint32_t)u), hi = dpp<CTRL>((uint32_t)(u >> 32));
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

__device__ inline double read_lane(double x, int lane)
{
    const uint64_t u = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

// The wave's sum, the same in every lane.
__device__ inline double wave_sum(double x)
{
    x += dpp_double<0x128>(x);
    x += dpp_double<0x124>(x);
    x += dpp_double<0x122>(x);
    x += dpp_double<0x121>(x);
    return (read_lane(x, 0) + read_lane(x, 16)) + (read_lane(x, 32) + read_lane(x, 48));
}

// ---------------------------------------------------------------------------
// Keys: numbers as unsigned integers of the same order, NaN above all, 0 for
// what cannot be chosen (no number maps to 0).
// ---------------------------------------------------------------------------
__device__ inline uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);   // -0 and +0 tie
    return x != x ? 0xffffffffu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ inline uint64_t order_key(double x)
{
    const uint64_t u = __double_as_longlong(x == 0.0 ? 0.0 : x);
    return x != x ? ~uint64_t(0) : (u >> 63) ? ~u : u | uint64_t(1) << 63;
}

// One round of a choice: the largest key of the wave and the lowest index
// that has it.  key is the lane's best key and at its index; the result is
// the same in every lane, found = false when all keys are 0.  The high
// words settle nearly every round; the low words and then the indices are
// compared only among lanes that tie so far.
__device__ inline bool wave_best(uint64_t key, int at, int &found_at)
{
    const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
    const uint32_t top = wave_max(hi);
    if (top == 0)
        return false;
    uint64_t tie = __ballot(hi == top);
    if (__popcll(tie) > 1) {
        const uint32_t low = wave_max(hi == top ? lo : 0u);
        tie = __ballot(hi == top && lo == low);
        if (__popcll(tie) > 1) {
            found_at = (int)~wave_max(hi == top && lo == low ? ~(uint32_t)at : 0u);
            return true;
        }
    }
    found_at = __builtin_amdgcn_readlane(at, (int)__builtin_ctzll(tie));
    return true;
}

// The row's largest logit among lanes' l[] (NaN ignored: the exponentials
// carry it), 0 for a row without any.
template <int V>
__device__ inline float row_max(const float (&l)[V])
{
    uint32_t best = order_key(-INFINITY);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (l[v] == l[v])
            best = max(best, order_key(l[v]));
    best = wave_max(best);
    const float m = __uint_as_float((best & 0x80000000u) ? best & 0x7fffffffu : ~best);
    return m == -INFINITY ? 0.f : m;
}

// Scores of the row, binary64.
template <int V>
__device__ inline void scores(const float (&l)[V], bool softmax, double (&s)[V])
{
    if (!softmax) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
        return;
    }
    const double m = row_max<V>(l);
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[v] = exp((double)l[v] - m);
        sum += s[v];
    }
    sum = wave_sum(sum);
    const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
    for (int v = 0; v < V; ++v)
        s[v] *= inv;
}

template <class E, int V>
__device__ inline void load_row(const typename E::T *row, int E_, int lane, float (&l)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * kWave + lane;
        l[v] = e < E_ ? (float)row[e] : -INFINITY;
    }
}

template <class E, int V>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs g)
{
    __shared__ double group_c[kRouteWaves][V * kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= g.T)
        return;                                      // whole waves; no barrier below
    const typename E::T *row = (const typename E::T *)g.logits + t * g.ldl;
    float l[V];
    load_row<E, V>(row, g.E, lane, l);
    const bool by_score = g.bias != nullptr;         // keys are c, else logits
    const bool need_s = by_score || g.groups > 1 || (g.softmax && !g.normalize);
    double s[V];
    if (need_s)
        scores<V>(l, g.softmax, s);

    uint64_t key[V];
    double c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * kWave + lane;
        const float b = by_score && e < g.E ? g.bias[e] : 0.f;
        c[v] = need_s ? s[v] + (double)b : 0.0;
        const bool there = e < g.E && l[v] != -INFINITY && b != -INFINITY;
        key[v] = !there ? 0 : by_score ? order_key(c[v]) : (uint64_t)order_key(l[v]) << 32;
    }

    if (g.groups > 1) {
        // Lane q sums the best of group q; it stays if fewer than
        // keep_groups groups come before it.
        const int per = g.E / g.groups;
        volatile double *mine = group_c[wave];       // the wave's own: written and read in program order
#pragma unroll
        for (int v = 0; v < V; ++v)
            mine[v * kWave + lane] = key[v] ? c[v] : -INFINITY;
        __builtin_amdgcn_wave_barrier();
        uint64_t score = 0;
        if (lane < g.groups) {
            double first = -INFINITY, second = -INFINITY;
            bool nan = false;
            for (int i = 0; i < per; ++i) {
                const double x = mine[lane * per + i];
                nan |= x != x;
                second = x > first ? first : x > second ? x : second;
                first = x > first ? x : first;
            }
            if (nan)
                score = ~uint64_t(0);
            else if (first != -INFINITY)
                score = order_key(first + (g.group_top > 1 && second != -INFINITY ? second : 0.0));
        }
        int before = 0;
        for (int q = 0; q < g.groups; ++q) {
            const uint64_t other = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(score >> 32), q) << 32 |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)score, q);
            before += other > score || (other == score && q < lane);
        }
        const uint64_t kept = __ballot(lane < g.groups && before < g.keep_groups);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * kWave + lane;
            if (e < g.E && !(kept >> (e / per) & 1))
                key[v] = 0;
        }
    }

    // k rounds; lane j keeps the j-th choice.
    int chosen = -1;
    for (int j = 0; j < g.k; ++j) {
        uint64_t best = key[0];
        int at = lane;
#pragma unroll
        for (int v = 1; v < V; ++v)
            if (key[v] > best) {
                best = key[v];
                at = v * kWave + lane;
            }
        int e;
        if (!wave_best(best, at, e))
            break;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * kWave + lane == e)
                key[v] = 0;
        if (lane == j)
            chosen = e;
    }

    // Weights of the chosen, a lane each.
    double w = 0.0;
    const float lj = chosen >= 0 ? (float)row[chosen] : -INFINITY;
    if (!g.softmax) {
        w = chosen >= 0 ? 1.0 / (1.0 + exp(-(double)lj)) : 0.0;
    } else if (g.normalize) {
        // softmax over the chosen alone: the other terms cancel
        const float one[1] = {lj};
        const double m = row_max<1>(one);
        w = chosen >= 0 ? exp((double)lj - m) : 0.0;
    } else {
        double sum = 0.0;                            // s of the chosen, from its owner
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double x = __shfl(s[v], chosen >= 0 ? chosen % kWave : 0);
            if (chosen >= 0 && chosen / kWave == v)
                sum = x;
        }
        w = sum;
    }
    if (g.normalize) {
        const double sum = wave_sum(w);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (lane < g.k) {
        g.index[t * g.k + lane] = chosen;
        g.weight[t * g.k + lane] = chosen >= 0 ? (float)(w * (double)g.scale) : 0.f;
    }
}

struct RouteGradArgs {
    const void *logits;
    const int *index;
    const float *dweight;
    void *dlogits;
    int64_t ldl, lddl;
    int T, E, k;
    bool softmax, normalize;
    float scale;
};

template <class E, int V>
__global__ __launch_bounds__(kRouteThreads) void route_grad_kernel(RouteGradArgs g)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= g.T)
        return;
    const typename E::T *row = (const typename E::T *)g.logits + t * g.ldl;
    typename E::T *out = (typename E::T *)g.dlogits + t * g.lddl;

    // Lane j holds the j-th choice.
    int chosen = lane < g.k ? g.index[t * g.k + lane] : -1;
    if (chosen < 0 || chosen >= g.E)
        chosen = -1;
    const double dw = chosen >= 0 ? (double)g.dweight[t * g.k + lane] * (double)g.scale : 0.0;
    const float lj = chosen >= 0 ? (float)row[chosen] : -INFINITY;

    double up;                                       // what the chosen logit gets
    double all = 0.0;                                // minus this times s(e) for every e
    double s[V];
    if (!g.softmax) {
        const double sj = chosen >= 0 ? 1.0 / (1.0 + exp(-(double)lj)) : 0.0;
        // 1 - s without cancellation
        const double rest = chosen >= 0 ? 1.0 / (1.0 + exp((double)lj)) : 0.0;
        if (g.normalize) {
            const double sum = wave_sum(sj);
            const double w = sum == 0.0 ? 0.0 : sj / sum;
            up = w * (dw - wave_sum(w * dw)) * rest;
        } else {
            up = sj * rest * dw;
        }
    } else if (g.normalize) {
        const float one[1] = {lj};
        const double m = row_max<1>(one);
        const double x = chosen >= 0 ? exp((double)lj - m) : 0.0;
        const double sum = wave_sum(x);
        const double w = sum == 0.0 ? 0.0 : x / sum;
        up = w * (dw - wave_sum(w * dw));
    } else {
        float l[V];
        load_row<E, V>(row, g.E, lane, l);
        scores<V>(l, true, s);
        double sj = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double x = __shfl(s[v], chosen >= 0 ? chosen % kWave : 0);
            if (chosen >= 0 && chosen / kWave == v)
                sj = x;
        }
        up = sj * dw;
        all = wave_sum(up);
    }

    double d[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        d[v] = g.softmax && !g.normalize ? -s[v] * all : 0.0;
    for (int j = 0; j < g.k; ++j) {
        const int e = __builtin_amdgcn_readlane(chosen, j);
        const double x = read_lane(up, j);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * kWave + lane == e)
                d[v] += x;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * kWave + lane;
        if (e < g.E)
            out[e] = (typename E::T)d[v];
    }
}

// ---------------------------------------------------------------------------
// Slot map
// ---------------------------------------------------------------------------
constexpr int kSlotThreads = 1024;
constexpr int kSlotWaves = kSlotThreads / kWave;
constexpr int kSlotChunk = 2048;                     // slots of a workgroup
constexpr int kSlotSteps = kSlotChunk / kSlotThreads;
static_assert(GEMM_F32_MAX_EXPERTS == kSlotThreads, "a thread per expert");

// counts[b][e]: slots of workgroup b's chunk that go to expert e.
__global__ __launch_bounds__(kSlotThreads) void count_slots(const int *index, int S, int E, int *counts)
{
    __shared__ int hist[GEMM_F32_MAX_EXPERTS];
    const int tid = threadIdx.x;
    hist[tid] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSlotChunk;
#pragma unroll
    for (int i = 0; i < kSlotSteps; ++i) {
        const int64_t s = first + i * kSlotThreads + tid;
        const int e = s < S ? index[s] : -1;
        if (e >= 0 && e < E)
            atomicAdd(&hist[e], 1);                  // LDS, whole numbers: any order
    }
    __syncthreads();
    if (tid < E)
        counts[(int64_t)blockIdx.x * E + tid] = hist[tid];
}

// Each workgroup places its chunk of kSlotChunk slots.  It needs, per expert, the slots
// of all chunks and of the chunks before its own: from counts, or (NULL) by
// counting all S slots itself, which needs no first launch.
// Wave w takes kSlotChunk / kSlotWaves slots, 64 at a time in rising order;
// base[w][e] is the next place of expert e for wave w.
__global__ __launch_bounds__(kSlotThreads) void place_slots(const int *index, int S, int E, const int *counts,
                                                            int *offsets, int *order, int *position)
{
    __shared__ int base[kSlotWaves][GEMM_F32_MAX_EXPERTS];
    __shared__ int others[2][GEMM_F32_MAX_EXPERTS];  // slots of the chunks before and behind
    __shared__ int wave_total[kSlotWaves];
    constexpr int kWaveSlots = kSlotChunk / kSlotWaves, kWaveSteps = kWaveSlots / kWave;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int64_t first = (int64_t)blockIdx.x * kSlotChunk;
#pragma unroll
    for (int w = 0; w < kSlotWaves; ++w)
        base[w][tid] = 0;
    others[0][tid] = others[1][tid] = 0;
    int mine[kWaveSteps];
#pragma unroll
    for (int i = 0; i < kWaveSteps; ++i) {
        const int64_t s = first + wave * kWaveSlots + i * kWave + lane;
        mine[i] = s < S ? index[s] : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaveSteps; ++i) {
        if (mine[i] >= E)
            mine[i] = -1;
        if (mine[i] >= 0)
            atomicAdd(&base[wave][mine[i]], 1);
    }
    int before = 0, total = 0;                       // of expert tid
    if (counts == nullptr) {
        constexpr int kBatch = 8;                    // loads in flight
        for (int64_t s0 = 0; s0 < S; s0 += kBatch * kSlotThreads) {
            int e[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int64_t s = s0 + q * kSlotThreads + tid;
                const bool own = s >= first && s < first + kSlotChunk;
                e[q] = s < S && !own ? index[s] : -1;
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                if (e[q] >= 0 && e[q] < E)
                    atomicAdd(&others[s0 + q * kSlotThreads >= first][e[q]], 1);   // chunks are whole multiples of the threads
        }
        __syncthreads();
        before = others[0][tid];
        total = before + others[1][tid];
    } else {
        if (tid < E) {
            constexpr int kBatch = 8;
            for (int b0 = 0; b0 < (int)gridDim.x; b0 += kBatch) {
                int n[kBatch];
#pragma unroll
                for (int q = 0; q < kBatch; ++q)
                    n[q] = b0 + q < (int)gridDim.x && b0 + q != (int)blockIdx.x ? counts[(int64_t)(b0 + q) * E + tid] : 0;
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    total += n[q];
                    before += b0 + q < (int)blockIdx.x ? n[q] : 0;
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int w = 0; w < kSlotWaves; ++w)
        total += base[w][tid];
    int scan = total;                                // inclusive over the wave
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int x = __shfl_up(scan, d);
        scan += lane >= d ? x : 0;
    }
    if (lane == kWave - 1)
        wave_total[wave] = scan;
    __syncthreads();
    int at = scan - total, placed = 0;
#pragma unroll
    for (int w = 0; w < kSlotWaves; ++w) {
        at += w < wave ? wave_total[w] : 0;
        placed += wave_total[w];
    }
    if (blockIdx.x == 0 && tid < E)
        offsets[tid] = at;
    if (blockIdx.x == 0 && tid == 0)
        offsets[E] = placed;
    int next_place = at + before;
#pragma unroll
    for (int w = 0; w < kSlotWaves; ++w) {
        const int n = base[w][tid];
        base[w][tid] = next_place;
        next_place += n;
    }
    __syncthreads();

    // Places: slots of one expert within 64 find each other bit by bit.
    volatile int *next = base[wave];                 // the wave's own from here on
#pragma unroll
    for (int i = 0; i < kWaveSteps; ++i) {
        const int e = mine[i];
        uint64_t same = __ballot(e >= 0);
        for (int bit = 1; bit < E; bit *= 2) {
            const uint64_t set = __ballot((e & bit) != 0);
            same &= (e & bit) ? set : ~set;
        }
        const int64_t s = first + wave * kWaveSlots + i * kWave + lane;
        int p = -1;
        if (e >= 0) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            p = next[e] + rank;
        }
        __builtin_amdgcn_wave_barrier();
        if (e >= 0) {
            if ((same >> lane) == 1)                 // the last of its expert
                next[e] = p + 1;
            order[p] = (int)s;
        }
        __builtin_amdgcn_wave_barrier();
        if (s < S) {
            position[s] = p;
            if (s >= placed)
                order[s] = -1;
        }
    }
}

int64_t slot_chunks(int64_t S) { return S <= kSlotChunk ? 1 : ceil_div(S, kSlotChunk); }

// Up to this many slots every workgroup counts them all; more are counted in a
// launch of their own.
constexpr int64_t kCountedInPlace = 1 << 17;

// A grid has fewer than 2^32 threads, a wave of them per token.
constexpr int kMaxTokens = (int)(UINT32_MAX / kWave) - kRouteWaves;

int check_route(int type, int T, int E, int k, int64_t ldl)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (T < 0 || T > kMaxTokens || E < 1 || E > GEMM_F32_MAX_EXPERTS || k < 1 || k > E || k > GEMM_F32_MAX_CHOSEN)
        return GEMM_F32_ERR_DIM;
    return ldl < E ? GEMM_F32_ERR_LD : GEMM_F32_OK;
}

// f(E{}, integral constant V) with 64 * V >= experts.
template <class E, class Fn>
void with_width(int experts, Fn &&f)
{
    if (experts <= 64)
        f(std::integral_constant<int, 1>{});
    else if (experts <= 128)
        f(std::integral_constant<int, 2>{});
    else if (experts <= 256)
        f(std::integral_constant<int, 4>{});
    else if (experts <= 512)
        f(std::integral_constant<int, 8>{});
    else
        f(std::integral_constant<int, 16>{});
}

}  // namespace
}  // namespace rows

using namespace rows;

extern "C" {

int gemm_f32_route(int type, int T, int E, int k, const void *logits, int ldl, const float *bias,
                   int score, int groups, int keep_groups, int group_top, int normalize, float scale,
                   float *weight, int *index, hipStream_t stream)
{
    const int rc = check_route(type, T, E, k, ldl);
    if (rc != GEMM_F32_OK)
        return rc;
    if ((score != GEMM_F32_SCORE_SOFTMAX && score != GEMM_F32_SCORE_SIGMOID) || groups < 1 ||
        groups > GEMM_F32_MAX_CHOSEN || E % groups != 0 || keep_groups < 1 || keep_groups > groups ||
        (group_top != 1 && group_top != 2))
        return GEMM_F32_ERR_OPTION;
    if (T == 0)
        return GEMM_F32_OK;
    if (logits == nullptr || weight == nullptr || index == nullptr)
        return GEMM_F32_ERR_NULL;
    if (!aligned_to(logits, type_bytes(type)) || !aligned_to(bias, 4) || !aligned_to(weight, 4) || !aligned_to(index, 4))
        return GEMM_F32_ERR_ALIGN;
    const RouteArgs g{logits, bias, weight, index, ldl, T, E, k, groups, keep_groups, group_top,
                      score == GEMM_F32_SCORE_SOFTMAX, normalize != 0, scale};
    const int grid = (int)ceil_div(T, kRouteWaves);
    with_type(type, [&](auto e) {
        using El = decltype(e);
        with_width<El>(E, [&](auto v) { route_kernel<El, v.value><<<grid, kRouteThreads, 0, stream>>>(g); });
    });
    return launched();
}

int gemm_f32_route_grad(int type, int T, int E, int k, const void *logits, int ldl, int score, int normalize,
                        float scale, const int *index, const float *dweight, void *dlogits, int lddl,
                        hipStream_t stream)
{
    const int rc = check_route(type, T, E, k, ldl < lddl ? ldl : lddl);
    if (rc != GEMM_F32_OK)
        return rc;
    if (score != GEMM_F32_SCORE_SOFTMAX && score != GEMM_F32_SCORE_SIGMOID)
        return GEMM_F32_ERR_OPTION;
    if (T == 0)
        return GEMM_F32_OK;
    if (logits == nullptr || index == nullptr || dweight == nullptr || dlogits == nullptr)
        return GEMM_F32_ERR_NULL;
    if (!aligned_to(logits, type_bytes(type)) || !aligned_to(dlogits, type_bytes(type)) || !aligned_to(index, 4) ||
        !aligned_to(dweight, 4))
        return GEMM_F32_ERR_ALIGN;
    const RouteGradArgs g{logits, index, dweight, dlogits, ldl, lddl, T, E, k,
                          score == GEMM_F32_SCORE_SOFTMAX, normalize != 0, scale};
    const int grid = (int)ceil_div(T, kRouteWaves);
    with_type(type, [&](auto e) {
        using El = decltype(e);
        with_width<El>(E, [&](auto v) { route_grad_kernel<El, v.value><<<grid, kRouteThreads, 0, stream>>>(g); });
    });
    return launched();
}

size_t gemm_f32_expert_map_ws_size(int S, int E)
{
    if (S < 0 || E < 1 || E > GEMM_F32_MAX_EXPERTS)
        return 0;
    return S > kCountedInPlace ? (size_t)slot_chunks(S) * (size_t)E * sizeof(int) : 0;
}

int gemm_f32_expert_map(int S, int E, const int *index, int *offsets, int *order, int *position, void *workspace,
                        size_t workspace_bytes, hipStream_t stream)
{
    if (S < 0 || E < 1 || E > GEMM_F32_MAX_EXPERTS)
        return GEMM_F32_ERR_DIM;
    if (offsets == nullptr || (S > 0 && (index == nullptr || order == nullptr || position == nullptr)))
        return GEMM_F32_ERR_NULL;
    if (!aligned_to(offsets, 4) || !aligned_to(index, 4) || !aligned_to(order, 4) || !aligned_to(position, 4))
        return GEMM_F32_ERR_ALIGN;
    const size_t need = gemm_f32_expert_map_ws_size(S, E);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned_to(workspace, 16)))
        return GEMM_F32_ERR_WORKSPACE;
    const int grid = (int)slot_chunks(S);
    int *counts = need > 0 ? (int *)workspace : nullptr;
    if (counts != nullptr)
        count_slots<<<grid, kSlotThreads, 0, stream>>>(index, S, E, counts);
    place_slots<<<grid, kSlotThreads, 0, stream>>>(index, S, E, counts, offsets, order, position);
    return launched();
}

}  // extern "C"
