// The gates' functions (include/gemm_f32_ffn.h), in binary32 for results that are rounded and
// in binary64 for decisions.
#ifndef GEMM_F32_FFN_GATE_H
#define GEMM_F32_FFN_GATE_H

#include "rows_common.h"

#include "gemm_f32_ffn.h"

namespace ffn {

using namespace rows;

inline bool known_gate(int gate) { return gate >= GEMM_F32_GATE_SILU && gate <= GEMM_F32_GATE_GELU_TANH; }

// Calls f(integral_constant) for the gate.
template <int V>
struct Gate {
    static constexpr int value = V;
};
template <class Fn>
inline void with_gate(int gate, Fn &&f)
{
    switch (gate) {
    case GEMM_F32_GATE_SILU: f(Gate<GEMM_F32_GATE_SILU>{}); break;
    case GEMM_F32_GATE_GELU: f(Gate<GEMM_F32_GATE_GELU>{}); break;
    case GEMM_F32_GATE_GELU_TANH: f(Gate<GEMM_F32_GATE_GELU_TANH>{}); break;
    default: f(Gate<GEMM_F32_GATE_NONE>{}); break;
    }
}

// e^-x for |x| up to 200, to a few steps of binary32: -x / ln 2 as a binary32 number and what its
// rounding lost, the first to the hardware's 2^x, the second to first order.  (The factors apart: the
// sigmoid adds 1 in the same step.)
__device__ inline void exp_minus(float x, float &power, float &factor)
{
    constexpr float kLog2e = 1.44269504089f, kLow = (float)(1.44269504088896340736 - (double)kLog2e), kLn2 = 0.69314718056f;
    const float high = x * -kLog2e, low = fmaf(x, -kLow, fmaf(x, -kLog2e, -high));
    power = __builtin_amdgcn_exp2f(high);
    factor = fmaf(low, kLn2, 1.f);
}
__device__ inline float exp_minus(float x)
{
    float power, factor;
    exp_minus(x, power, factor);
    return power * factor;
}

// 1 / (1 + e^-x).  Clamped: e^-100 adds nothing to 1, and e^200 is an infinity.
__device__ inline float sigmoid(float x)
{
    float power, factor;
    exp_minus(__builtin_amdgcn_fmed3f(x, -200.f, 100.f), power, factor);
    return __builtin_amdgcn_rcpf(fmaf(power, factor, 1.f));
}
// s = 1 / (1 + e^-x) and 1 - s, without cancellation on either side.
__device__ inline void sigmoid(float x, float &s, float &rest)
{
    const float e = exp_minus(fminf(fabsf(x), 200.f)), r = __builtin_amdgcn_rcpf(1.f + e);
    s = x < 0.f ? e * r : r;
    rest = x < 0.f ? r : e * r;
}

// gelu_tanh(g) = g / (1 + e^-v), v = g (kA + kB g^2), because (1 + tanh(v/2)) / 2 is the sigmoid of v.
constexpr double kA = 1.59576912160573071176, kB = kA * 0.044715;     // sqrt(8 / pi)

// p(g) = (1 + erf(g / sqrt 2)) / 2 = e^(-g^2 / 2) erfcx(|g| / sqrt 2) / 2 on the left, 1 less that on the right.
// erfcx(z) / 2 for z = 0 .. 9.6 (further on the exponential is 0) is a polynomial in t = 1 / (1 + 0.4 z), fitted
// to its relative error by reweighted least squares on Chebyshev nodes: 6e-8 off, 4e-7 in binary32.  (The
// library's erfcf took twice the time of the 8-bit rows' whole kernel without it.)
// power: e^(-g^2 / 2).
__device__ inline float gelu_part(float g, float &power)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.28284271247f, 1.f));
    float q = 0.0202376172f;
    q = fmaf(q, t, -0.068247743f);
    q = fmaf(q, t, 0.0379958786f);
    q = fmaf(q, t, 0.0486143343f);
    q = fmaf(q, t, 0.0366340727f);
    q = fmaf(q, t, 0.098099038f);
    q = fmaf(q, t, 0.100579329f);
    q = fmaf(q, t, 0.113273494f);
    q = fmaf(q, t, 0.112814017f);
    power = exp_minus(fminf(0.5f * g * g, 200.f));
    const float tail = q * t * power;
    return g < 0.f ? tail : 1.f - tail;
}

template <int GATE>
__device__ inline float gate(float g)
{
    if constexpr (GATE == GEMM_F32_GATE_SILU) {
        return g * sigmoid(g);
    } else if constexpr (GATE == GEMM_F32_GATE_GELU) {
        float power;
        return g * gelu_part(g, power);
    } else {
        return g * sigmoid(g * fmaf((float)kB * g, g, (float)kA));
    }
}

// The gate's value and derivative.
template <int GATE>
__device__ inline void gate_slope(float g, float &value, float &slope)
{
    if constexpr (GATE == GEMM_F32_GATE_SILU) {
        float s, rest;
        sigmoid(g, s, rest);
        value = g * s;
        slope = s * fmaf(g, rest, 1.f);
    } else if constexpr (GATE == GEMM_F32_GATE_GELU) {
        float power;
        const float p = gelu_part(g, power);
        value = g * p;
        slope = fmaf(g * 0.39894228040f, power, p);
    } else {
        float s, rest;
        sigmoid(g * fmaf((float)kB * g, g, (float)kA), s, rest);
        value = g * s;
        // s (1 - s) is 0 long before |g| = 32: the clamp keeps g^2 from an infinity times that
        const float c = g > 32.f ? 32.f : g < -32.f ? -32.f : g;
        slope = fmaf(c * s, rest * fmaf((float)(3 * kB) * c, c, (float)kA), s);
    }
}

template <int GATE>
__device__ inline double gate64(double g)
{
    if constexpr (GATE == GEMM_F32_GATE_SILU)
        return g / (1.0 + exp(-g));
    else if constexpr (GATE == GEMM_F32_GATE_GELU)
        return 0.5 * g * erfc(g * -0.70710678118654752440);
    else
        return g / (1.0 + exp(-g * fma(kB * g, g, kA)));
}

// How far gate<GATE>(g) may be off, relative.  silu: the exponential's few steps.  The others have an argument
// (g^2 / 2, or v) whose rounding counts as often as it is large: 8 and 11 at g = -4, 90 where the result stops
// being a normal number; on the right the exponential itself is small beside 1.
constexpr float kGateFar = 0x1p-15f;
template <int GATE>
__device__ inline float gate_error(float g)
{
    return GATE == GEMM_F32_GATE_SILU ? 0x1p-20f : g < -4.f ? kGateFar : 0x1p-18f;
}

}  // namespace ffn

#endif
