// activation.cuh -- the activations of the feed-forward layers and their slopes, in fp32.
//
// Each is written as z times a factor in [0, 1]: its tail stays accurate where 1 + erf or
// 1 + tanh would cancel, until it falls below 2^-126 and is 0 (silu: z < -87, gelu: -13, its tanh form: -10).
// z enters that product no lower than -FLT_MAX and the factor's slope within +-1e6 (where it has long
// vanished), so that no infinity meets a zero; a NaN stays one.
#pragma once

#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace gemmar {

// == GEMMAR_ACT_*
enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + exp(-z)); the divisor is at least 1, and an infinite one gives 0.  The fast exponential rounds
// z / ln 2 once, which costs (2 + |z|) 2^-24 of its value: less than the sums before it.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
constexpr float kLowest = -3.402823466e38f;

// The argument of the tanh form's sigmoid ((1 + tanh u) / 2 = sigmoid(2 u))
__device__ __forceinline__ float tanh_arg(float z) { return 2.0f * kSqrt2OverPi * z * fmaf(kGeluCubic * z, z, 1.0f); }

// The coefficient of t^(9-i) in P, below.
__device__ __forceinline__ constexpr float cdf_term(int i)
{
    constexpr float c[10] = {-2.062856220e-02f, 1.124642864e-01f, -2.282836586e-01f, 1.918818653e-01f, -7.950805128e-02f,
                             9.620437026e-02f,  7.837239653e-02f, 1.102393121e-01f,  1.195713207e-01f, 1.196867153e-01f};
    return c[i];
}

// Phi(z), and e = exp(-z^2 / 2).  Phi(-a) = e t P(t) for a >= 0 with t = 1 / (1 + 0.3 a), in which the
// rest is smooth down to t = 0, and P of degree 9, fitted here to a relative 4e-9 for a up to 15 (weighted
// least squares in 40 digits, reweighted towards equal errors).  The whole is off by (3 + z^2 / 2) 2^-23 of
// its value (the exponential's argument is rounded twice), in either tail.
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float a = fabsf(z);
    e = __expf(-0.5f * a * a);
    const float t = __fdividef(1.0f, fmaf(0.3f, a, 1.0f));   // 0 for the largest a, as is e
    float p = cdf_term(0);
#pragma unroll
    for (int i = 1; i < 10; ++i)
        p = fmaf(p, t, cdf_term(i));
    const float tail = p * t * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == ACT_RELU)
        return max_nan(z, 0.0f);
    if constexpr (ACT == ACT_SILU)
        return max_nan(z, kLowest) * sigmoid(z);
    if constexpr (ACT == ACT_GELU_TANH)
        return max_nan(z, kLowest) * sigmoid(tanh_arg(z));
    if constexpr (ACT == ACT_GELU) {
        float e;
        return max_nan(z, kLowest) * normal_cdf(z, e);
    }
    return z;
}

// gelu of W values by a warp that has its scheduler to itself: through eight values at a time, two an
// instruction (a 128 x 256 tile's finish with one after another takes 3 us more).
template <int W>
__device__ __forceinline__ void gelu_values(float (&v)[W])
{
    constexpr int G = 8;
    static_assert(W % G == 0, "groups");
#pragma unroll
    for (int g = 0; g < W; g += G) {
        float t[G], e[G], p[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const float a = fabsf(v[g + i]);
            t[i] = __fdividef(1.0f, fmaf(0.3f, a, 1.0f));
            e[i] = __expf(-0.5f * a * a);
            p[i] = cdf_term(0);
        }
#pragma unroll
        for (int k = 1; k < 10; ++k)
#pragma unroll
            for (int i = 0; i < G; i += 2) {
                float x = cdf_term(k), y = x;
                ptx::fma2(x, y, p[i], p[i + 1], t[i], t[i + 1]);
                p[i] = x;
                p[i + 1] = y;
            }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const float tail = p[i] * t[i] * e[i];
            v[g + i] = max_nan(v[g + i], kLowest) * (v[g + i] < 0.0f ? tail : 1.0f - tail);
        }
    }
}

// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ void act_slope(float z, float &value, float &slope)
{
    value = z;
    slope = 1.0f;
    if constexpr (ACT == ACT_RELU) {
        value = max_nan(z, 0.0f);
        slope = z > 0.0f ? 1.0f : min_nan(value, 0.0f);   // 0, or the NaN
    }
    if constexpr (ACT == ACT_SILU || ACT == ACT_GELU_TANH || ACT == ACT_GELU) {
        const float c = max_nan(min_nan(z, 1e6f), -1e6f);
        float s, d;   // the factor, and its slope
        if constexpr (ACT == ACT_SILU) {
            s = sigmoid(z);
            d = fmaf(-s, s, s);
        } else if constexpr (ACT == ACT_GELU_TANH) {
            s = sigmoid(tanh_arg(z));
            d = fmaf(-s, s, s) * (2.0f * kSqrt2OverPi * fmaf(3.0f * kGeluCubic * c, c, 1.0f));
        } else {
            s = normal_cdf(z, d);
            d *= 0.3989422804f;
        }
        value = max_nan(z, kLowest) * s;
        slope = fmaf(c, d, s);
    }
}

// f with the activation as a compile-time value: one branch for all the elements f handles
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>()); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>()); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>()); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, ACT_NONE>()); break;
    }
}

}  // namespace gemmar
