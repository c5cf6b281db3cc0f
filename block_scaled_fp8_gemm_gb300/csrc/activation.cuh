// activation.cuh -- the activations of the feed-forward layers and their slopes, in fp32.
//
// Each is written as z times a factor in [0, 1] (its tail stays accurate where 1 + erf or
// 1 + tanh would cancel), and where that factor or its slope has vanished the limit is
// returned instead of a product with an infinity.
#pragma once

#include <cstdint>
#include <type_traits>

namespace gemmar {

// == GEMMAR_ACT_*
enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_COUNT = 5 };

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + exp(-z)); the divisor is at least 1, and an infinite one gives 0.  The fast exponential rounds
// z / ln 2 once, which costs (2 + |z|) 2^-24 of its value: less than the sums before it.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == ACT_RELU)
        return z < 0.0f ? 0.0f : z;   // a NaN stays one
    if constexpr (ACT == ACT_SILU || ACT == ACT_GELU_TANH || ACT == ACT_GELU) {
        float s;
        if constexpr (ACT == ACT_SILU)
            s = sigmoid(z);
        else if constexpr (ACT == ACT_GELU_TANH)   // (1 + tanh u) / 2 = sigmoid(2 u)
            s = sigmoid(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
        else
            s = 0.5f * erfcf(-0.70710678f * z);
        return s == 0.0f ? 0.0f : z * s;
    }
    return z;
}

// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ void act_slope(float z, float &value, float &slope)
{
    value = z;
    slope = 1.0f;
    if constexpr (ACT == ACT_RELU) {
        value = z < 0.0f ? 0.0f : z;
        slope = z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    }
    if constexpr (ACT == ACT_SILU || ACT == ACT_GELU_TANH) {
        // value = z s(v), slope = s + z s (1 - s) v'
        float v = z, dv = 1.0f;
        if constexpr (ACT == ACT_GELU_TANH) {
            const float z2 = z * z;
            v = 2.0f * kSqrt2OverPi * (z + kGeluCubic * z2 * z);
            dv = 2.0f * kSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z2);
        }
        const float s = sigmoid(v), t = s * (1.0f - s);
        value = s == 0.0f ? 0.0f : z * s;
        slope = t == 0.0f ? s : s + z * t * dv;
    }
    if constexpr (ACT == ACT_GELU) {
        const float s = 0.5f * erfcf(-0.70710678f * z), d = 0.3989422804f * expf(-0.5f * z * z);
        value = s == 0.0f ? 0.0f : z * s;
        slope = d == 0.0f ? s : s + z * d;
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
