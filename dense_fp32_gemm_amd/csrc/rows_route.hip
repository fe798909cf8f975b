// Routing of tokens to experts, its gradient, and the slot map
// (include/gemm_f32_rows.h).
//
//  * route_kernel: 16 or 64 lanes per token, each with every 16th (64th) expert; the
//    choice is k rounds of a maximum over integer keys.
//  * route_grad_kernel: the same layout.
//  * count_slots, sum_counts, place_slots: a stable counting sort of the slots by expert,
//    a workgroup per kSlotChunk slots.
//
// Scores are binary64: which expert is taken hangs on differences between
// neighbouring scores, and a score rounded to 24 bits makes ties (and with
// them wrong choices) of what the formula tells apart.

#include <type_traits>

#include "rows_common.h"

namespace rows {
namespace {

constexpr int kRouteWaves = 4;
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
    Divisor per_group;
};

// ---------------------------------------------------------------------------
// L lanes (16 or 64) share a token; lane i of them holds experts i, i + L, ...
// Reductions over the token's lanes give every one of them the result.
// ---------------------------------------------------------------------------
template <int L, class Fn>
__device__ inline uint32_t reduce(uint32_t x, Fn &&f)
{
    x = f(x, dpp<0x128>(x));     // rotations within 16 lanes
    x = f(x, dpp<0x124>(x));
    x = f(x, dpp<0x122>(x));
    x = f(x, dpp<0x121>(x));
    if constexpr (L == 64) {
        x = f(x, (uint32_t)__shfl_xor((int)x, 16));
        x = f(x, (uint32_t)__shfl_xor((int)x, 32));
    }
    return x;
}
template <int L>
__device__ inline uint32_t token_max(uint32_t x)
{
    return reduce<L>(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L>
__device__ inline uint32_t token_min(uint32_t x)
{
    return reduce<L>(x, [](uint32_t a, uint32_t b) { return min(a, b); });
}

template <int CTRL>
__device__ inline double dpp_double(double x)
{
    const uint64_t u = __double_as_longlong(x);
    const uint32_t lo = dpp<CTRL>((uint32_t)u), hi = dpp<CTRL>((uint32_t)(u >> 32));
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

template <int L>
__device__ inline double token_sum(double x)
{
    x += dpp_double<0x128>(x);
    x += dpp_double<0x124>(x);
    x += dpp_double<0x122>(x);
    x += dpp_double<0x121>(x);
    if constexpr (L == 64) {
        x += __shfl_xor(x, 16);
        x += __shfl_xor(x, 32);
    }
    return x;
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

// The token's largest key among its lanes' best ones.
template <int L>
__device__ inline uint32_t top_key(uint32_t best) { return token_max<L>(best); }
template <int L>
__device__ inline uint64_t top_key(uint64_t best)
{
    const uint32_t hi = token_max<L>((uint32_t)(best >> 32));
    const uint32_t lo = token_max<L>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The row's largest logit among lanes' l[] (NaN ignored: the exponentials
// carry it), 0 for a row without any.
template <int L, int V>
__device__ inline float row_max(const float (&l)[V])
{
    uint32_t best = order_key(-INFINITY);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (l[v] == l[v])
            best = max(best, order_key(l[v]));
    best = token_max<L>(best);
    const float m = __uint_as_float((best & 0x80000000u) ? best & 0x7fffffffu : ~best);
    return m == -INFINITY ? 0.f : m;
}

// Scores of the row, binary64.
template <int L, int V>
__device__ inline void scores(const float (&l)[V], bool softmax, double (&s)[V])
{
    if (!softmax) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
        return;
    }
    const double m = row_max<L, V>(l);
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[v] = exp((double)l[v] - m);
        sum += s[v];
    }
    sum = token_sum<L>(sum);
    const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
    for (int v = 0; v < V; ++v)
        s[v] *= inv;
}

template <class E, int L, int V>
__device__ inline void load_row(const typename E::T *row, int experts, int i, float (&l)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * L + i;
        l[v] = e < experts ? (float)row[e] : -INFINITY;
    }
}

// s of expert e, from the lane of the token that holds it.
template <int L, int V>
__device__ inline double score_of(const double (&s)[V], int e)
{
    double x = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const double y = __shfl(s[v], e >= 0 ? e % L : 0, L);
        x = e >= 0 && e / L == v ? y : x;
    }
    return x;
}

// k rounds: the largest key of the token, of those the lowest expert; lane j of
// the token gets the j-th choice (-1: none), k <= L.
template <int L, int V, class Key>
__device__ inline int choose(Key (&key)[V], int k, int i)
{
    int chosen = -1;
    for (int j = 0; j < k; ++j) {
        Key best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            best = key[v] > best ? key[v] : best;
        const Key top = top_key<L>(best);
        uint32_t at = UINT32_MAX;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            at = key[v] == top ? (uint32_t)(v * L + i) : at;
        at = token_min<L>(at);
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = (uint32_t)(v * L + i) == at ? 0 : key[v];
        chosen = i == j && top != 0 ? (int)at : chosen;
    }
    return chosen;
}

// KEY64: keys are c (a bias), else the logits'.  Bound by latency and by the binary64
// exponentials: 16384 x 128 bf16 logits without a bias take 8.2 us (0.6 TB/s of
// their 5.2 MB), 8192 x 256 binary32 with one and with groups, a sigmoid of every
// logit, 19 us.
template <class E, int L, int V, bool KEY64>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs g)
{
    constexpr int R = kWave / L, kPad = 32;          // tokens of a wave; experts between gaps of one in LDS
    constexpr int kLine = L * V + L * V / kPad + 1;
    __shared__ double group_c[kRouteWaves][R][kLine];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int i = lane % L, r = lane / L;
    const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * R;
    if (t0 >= g.T)
        return;                                      // whole waves; no barrier below
    const bool live = t0 + r < g.T;                  // lanes past the last token work on a copy of it
    const int64_t t = live ? t0 + r : g.T - 1;
    const typename E::T *row = (const typename E::T *)g.logits + t * g.ldl;
    float l[V];
    load_row<E, L, V>(row, g.E, i, l);
    const bool need_s = KEY64 || g.groups > 1 || (g.softmax && !g.normalize);
    double s[V], c[V];
    if (need_s)
        scores<L, V>(l, g.softmax, s);

    using Key = typename std::conditional<KEY64, uint64_t, uint32_t>::type;
    Key key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * L + i;
        const float b = KEY64 && e < g.E ? g.bias[e] : 0.f;
        c[v] = need_s ? s[v] + (double)b : 0.0;
        const bool there = e < g.E && l[v] != -INFINITY && b != -INFINITY;
        if constexpr (KEY64)
            key[v] = there ? order_key(c[v]) : 0;
        else
            key[v] = there ? order_key(l[v]) : 0;
    }

    if (g.groups > 1) {
        // Lane q sums the best of group q; it stays if fewer than
        // keep_groups groups come before it.
        const int per = g.E / g.groups;
        volatile double *mine = group_c[wave][r];    // the wave's own: written and read in program order
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * L + i;
            mine[e + e / kPad] = key[v] ? c[v] : -INFINITY;
        }
        __builtin_amdgcn_wave_barrier();
        uint64_t score = 0;
        if (i < g.groups) {
            double first = -INFINITY, second = -INFINITY;
            bool nan = false;
            for (int q = 0; q < per; ++q) {
                const int e = i * per + q;
                const double x = mine[e + e / kPad];
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
            const uint64_t other = (uint64_t)(uint32_t)__shfl((int)(score >> 32), q, L) << 32 |
                                   (uint32_t)__shfl((int)(uint32_t)score, q, L);
            before += other > score || (other == score && q < i);
        }
        const uint64_t kept = __ballot(i < g.groups && before < g.keep_groups) >> (r * L);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * L + i;
            if (e < g.E && !(kept >> g.per_group.of(e) & 1))
                key[v] = 0;
        }
    }
    const int chosen = choose<L, V>(key, g.k, i);

    // Weights of the chosen, a lane each.
    double w = 0.0;
    const float lj = chosen >= 0 ? (float)row[chosen] : -INFINITY;
    if (!g.softmax) {
        w = chosen >= 0 ? 1.0 / (1.0 + exp(-(double)lj)) : 0.0;
    } else if (g.normalize) {
        // softmax over the chosen alone: the other terms cancel
        const float one[1] = {lj};
        const double m = row_max<L, 1>(one);
        w = chosen >= 0 ? exp((double)lj - m) : 0.0;
    } else {
        w = score_of<L, V>(s, chosen);
    }
    if (g.normalize) {
        const double sum = token_sum<L>(w);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (live && i < g.k) {
        g.index[t * g.k + i] = chosen;
        g.weight[t * g.k + i] = chosen >= 0 ? (float)(w * (double)g.scale) : 0.f;
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

// Bound like route_kernel: 16384 x 128 bf16, k = 8, 7.5 us (1.1 TB/s of 8.4 MB).
template <class E, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_grad_kernel(RouteGradArgs g)
{
    constexpr int R = kWave / L;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int i = lane % L, r = lane / L;
    const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * R;
    if (t0 >= g.T)
        return;
    const bool live = t0 + r < g.T;
    const int64_t t = live ? t0 + r : g.T - 1;
    const typename E::T *row = (const typename E::T *)g.logits + t * g.ldl;
    typename E::T *out = (typename E::T *)g.dlogits + t * g.lddl;

    // Lane j holds the j-th choice.
    int chosen = i < g.k ? g.index[t * g.k + i] : -1;
    if (chosen < 0 || chosen >= g.E)
        chosen = -1;
    const double dw = chosen >= 0 ? (double)g.dweight[t * g.k + i] * (double)g.scale : 0.0;
    const float lj = chosen >= 0 ? (float)row[chosen] : -INFINITY;

    double up;                                       // what the chosen logit gets
    double all = 0.0;                                // minus this times s(e) for every e
    double s[V];
    if (!g.softmax) {
        const double sj = chosen >= 0 ? 1.0 / (1.0 + exp(-(double)lj)) : 0.0;
        // 1 - s without cancellation
        const double rest = chosen >= 0 ? 1.0 / (1.0 + exp((double)lj)) : 0.0;
        if (g.normalize) {
            const double sum = token_sum<L>(sj);
            const double w = sum == 0.0 ? 0.0 : sj / sum;
            up = w * (dw - token_sum<L>(w * dw)) * rest;
        } else {
            up = sj * rest * dw;
        }
    } else if (g.normalize) {
        const float one[1] = {lj};
        const double m = row_max<L, 1>(one);
        const double x = chosen >= 0 ? exp((double)lj - m) : 0.0;
        const double sum = token_sum<L>(x);
        const double w = sum == 0.0 ? 0.0 : x / sum;
        up = w * (dw - token_sum<L>(w * dw));
    } else {
        float l[V];
        load_row<E, L, V>(row, g.E, i, l);
        scores<L, V>(l, true, s);
        up = score_of<L, V>(s, chosen) * dw;
        all = token_sum<L>(up);
    }

    double d[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        d[v] = g.softmax && !g.normalize ? -s[v] * all : 0.0;
    for (int j = 0; j < g.k; ++j) {
        const int e = __shfl(chosen, j, L);
        const double x = __shfl(up, j, L);
#pragma unroll
        for (int v = 0; v < V; ++v)
            d[v] += v * L + i == e ? x : 0.0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * L + i;
        if (live && e < g.E)
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

// counts[b][e] becomes the slots of expert e in the chunks before b, counts[chunks][e]
// those in all of them.  A workgroup per 64 experts, a wave per part of the chunks.
__global__ __launch_bounds__(kSlotThreads) void sum_counts(int *counts, int chunks, int E)
{
    __shared__ int part[kSlotWaves][kWave];
    constexpr int kBatch = 8;                        // loads in flight
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int e = blockIdx.x * kWave + lane;
    const int64_t each = (chunks + kSlotWaves - 1) / kSlotWaves;
    const int64_t first = wave * each, last = first + each < chunks ? first + each : chunks;
    int n[kBatch];
    auto load = [&](int64_t b0) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            n[q] = e < E && b0 + q < last ? counts[(b0 + q) * E + e] : 0;
    };
    int sum = 0;
    for (int64_t b0 = first; b0 < last; b0 += kBatch) {
        load(b0);
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            sum += n[q];
    }
    part[wave][lane] = sum;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSlotWaves; ++w) {
        before += w < wave ? part[w][lane] : 0;
        total += part[w][lane];
    }
    for (int64_t b0 = first; b0 < last; b0 += kBatch) {
        load(b0);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (e < E && b0 + q < last)
                counts[(b0 + q) * E + e] = before;
            before += n[q];
        }
    }
    if (wave == 0 && e < E)
        counts[(int64_t)chunks * E + e] = total;
}

// Each workgroup places its chunk of kSlotChunk slots.  It needs, per expert, the slots
// of all chunks and of the chunks before its own: from counts (`summed`: from
// sums of them), or (NULL) by counting all S slots itself, which needs no first launch.
// 65536 slots 7.8 us, 131072 9.6 us: chains of LDS atomics and ballots, no bandwidth.
// Wave w takes kSlotChunk / kSlotWaves slots, 64 at a time in rising order;
// base[w][e] is the next place of expert e for wave w.
__global__ __launch_bounds__(kSlotThreads) void place_slots(const int *index, int S, int E, const int *counts,
                                                            bool summed, int *offsets, int *order, int *position)
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
        if (tid < E && summed) {
            before = counts[(int64_t)blockIdx.x * E + tid];
            total = counts[(int64_t)gridDim.x * E + tid];
        } else if (tid < E) {
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
    if (!summed) {
#pragma unroll
        for (int w = 0; w < kSlotWaves; ++w)
            total += base[w][tid];
    }
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
// launch of their own (16384 slots: 7.7 us in one launch; 65536: 14 us against 10 in
// two, 131072: 23 against 12).
constexpr int64_t kCountedInPlace = 1 << 15;
// From this many chunks on their counts are summed in a launch of their own; fewer,
// and every workgroup of the last launch adds them up itself.  That work grows with the square
// of the slots (in a graph, us without and with the third launch: 65536 slots 9.9 and 11.4,
// 262144: 16.6 and 12.8, 1048576: 46 and 22, 16777216: 7600 and 214); the launch costs a caller
// outside of a graph up to 3 us.  In between, where the one loses what the other gains, the limit is
// for the caller without a graph (131072 slots, E = 64: 13.7 and 16.3, in a graph 11.2 and 11.0;
// 196608 slots, E = 64: 14.0 and 16.7, in a graph 13.5 and 11.4, E = 256: 15.0 and 16.7, in a graph 14.8 and 12.1).
constexpr int64_t kSummedFrom = 128;

// A grid has fewer than 2^32 threads, a wave of them per token.
constexpr int kMaxTokens = (int)(UINT32_MAX / kWave) - kRouteWaves;

// Tokens from which 16 lanes take one of more than 128 experts.
constexpr int kNarrowFrom = 4096;

int check_route(int type, int T, int E, int k, int64_t ldl)
{
    if (!known_type(type))
        return GEMM_F32_ERR_TYPE;
    if (T < 0 || T > kMaxTokens || E < 1 || E > GEMM_F32_MAX_EXPERTS || k < 1 || k > E || k > GEMM_F32_MAX_CHOSEN)
        return GEMM_F32_ERR_DIM;
    return ldl < E ? GEMM_F32_ERR_LD : GEMM_F32_OK;
}

// f(L, V, tokens of a workgroup) for the lanes of a token and the experts of a
// lane, as integral constants.  16 lanes a token (four tokens a wave) need a quarter of
// the instructions of a choice; 64 where the experts, the choices or the groups are too
// many for them, and where tokens are too few to fill the device's waves (512 tokens,
// 256 experts, bias and groups: 11.7 us against 14.8; 8192 tokens: 24 against 18; 16383
// tokens, 128 experts, no bias: 16.7 against 7.6; 256 tokens, 128 experts: 5.6 against 4.4).
template <class Fn>
void with_width(int T, int experts, int most, Fn &&f)
{
    auto wide = [&](auto v) { f(std::integral_constant<int, 64>{}, v, kRouteWaves); };
    auto narrow = [&](auto v) { f(std::integral_constant<int, 16>{}, v, kRouteWaves * 4); };
    if (most <= 16 && (experts <= 128 || (experts <= 256 && T >= kNarrowFrom))) {
        if (experts <= 64)
            narrow(std::integral_constant<int, 4>{});
        else if (experts <= 128)
            narrow(std::integral_constant<int, 8>{});
        else
            narrow(std::integral_constant<int, 16>{});
    } else if (experts <= 64) {
        wide(std::integral_constant<int, 1>{});
    } else if (experts <= 256) {
        wide(std::integral_constant<int, 4>{});
    } else {
        wide(std::integral_constant<int, 16>{});
    }
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
                      score == GEMM_F32_SCORE_SOFTMAX, normalize != 0, scale, Divisor(E / groups)};
    with_type(type, [&](auto e) {
        using El = decltype(e);
        with_width(T, E, k > groups ? k : groups, [&](auto lanes, auto v, int tokens) {
            const int grid = (int)ceil_div(T, tokens);
            if (bias != nullptr)
                route_kernel<El, lanes.value, v.value, true><<<grid, kRouteThreads, 0, stream>>>(g);
            else
                route_kernel<El, lanes.value, v.value, false><<<grid, kRouteThreads, 0, stream>>>(g);
        });
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
    with_type(type, [&](auto e) {
        using El = decltype(e);
        with_width(T, E, k, [&](auto lanes, auto v, int tokens) {
            route_grad_kernel<El, lanes.value, v.value><<<(int)ceil_div(T, tokens), kRouteThreads, 0, stream>>>(g);
        });
    });
    return launched();
}

size_t gemm_f32_expert_map_ws_size(int S, int E)
{
    if (S < 0 || E < 1 || E > GEMM_F32_MAX_EXPERTS)
        return 0;
    return S > kCountedInPlace ? (size_t)(slot_chunks(S) + 1) * (size_t)E * sizeof(int) : 0;
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
    const bool summed = counts != nullptr && grid >= kSummedFrom;
    if (summed)
        sum_counts<<<(int)ceil_div(E, kWave), kSlotThreads, 0, stream>>>(counts, grid, E);
    place_slots<<<grid, kSlotThreads, 0, stream>>>(index, S, E, counts, summed, offsets, order, position);
    return launched();
}

}  // extern "C"
