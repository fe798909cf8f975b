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

// e^-a for a >= 0 (0 past 200), to a few steps of binary32: -a / ln 2 as a binary32 number
// and what its rounding lost, the first to the hardware's 2^x, the second to first order.
__device__ inline float exp_minus(float a)
{
    constexpr float kLog2e = 1.44269504089f, kLow = (float)(1.44269504088896340736 - (double)kLog2e), kLn2 = 0.69314718056f;
    a = fminf(a, 200.f);
    const float high = a * -kLog2e, low = fmaf(a, -kLog2e, -high) - a * kLow;
    return __builtin_amdgcn_exp2f(high) * fmaf(low, kLn2, 1.f);
}

// s = 1 / (1 + e^-x) and 1 - s, without cancellation on either side.
__device__ inline void sigmoid(float x, float &s, float &rest)
{
    const float e = exp_minus(fabsf(x)), r = __builtin_amdgcn_rcpf(1.f + e);
    s = x < 0.f ? e * r : r;
    rest = x < 0.f ? r : e * r;
}

// gelu_tanh(g) = g / (1 + e^-v), v = g (kA + kB g^2), because (1 + tanh(v/2)) / 2 is the sigmoid of v.
constexpr double kA = 1.59576912160573071176, kB = kA * 0.044715;     // sqrt(8 / pi)

template <int GATE>
__device__ inline float gate(float g)
{
    if constexpr (GATE == GEMM_F32_GATE_SILU) {
        float s, rest;
        sigmoid(g, s, rest);
        return g * s;
    } else if constexpr (GATE == GEMM_F32_GATE_GELU) {
        return 0.5f * g * erfcf(g * -0.70710678119f);                   // erfc: no cancellation for g < 0
    } else {
        float s, rest;
        sigmoid(g * fmaf((float)kB * g, g, (float)kA), s, rest);
        return g * s;
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
        const float p = 0.5f * erfcf(g * -0.70710678119f);
        value = g * p;
        slope = fmaf(g * 0.39894228040f, exp_minus(0.5f * g * g), p);
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

// How far gate<GATE>() may be off, relative: the argument's rounding (and that of v and g^2 / 2,
// which are up to about 90 where the result is a normal number) times the function's own growth there, and a few steps.
template <int GATE>
constexpr float gate_error()
{
    return GATE == GEMM_F32_GATE_SILU ? 0x1p-20f : 0x1p-15f;
}

}  // namespace ffn

#endif
