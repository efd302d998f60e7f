// Activations of the linear layers with their slopes, in FP32. EXACT: for FP32
// results, on CUDA's exponential and normal distribution functions; else for results that are
// rounded to bfloat16, on the hardware's 2^x and 1 / x (relative errors of 2^-22), with
// the normal distribution's tail as its density times a polynomial, which costs a
// third. The polynomial, in t = 1 / (1 + 0.495 a) as in Hastings' approximations of erf
// for a = |z| / sqrt(2), was fitted to exp(a^2) erfc(a) by linear programming: off by less than
// 2^-11 of itself up to a = 9.6, where the density leaves FP32, and the distribution
// by 7e-7. (A fit of the distribution's error alone, 1.5e-7, is 1 % off at z = -8, more than a
// rounding to bfloat16; a degree more holds both, 2^-13 and 5e-8, but 4096 x 16384 x 4096
// then takes 359 us for 355.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgemm_linear.h"

namespace sgemm_dev {

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_whole(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z)
{
    if constexpr (EXACT)  // (1 / x to 2^-23 of itself; below 2^-126 too)
        return rcp_whole(1.0f + expf(-z));
    else
        return rcp(1.0f + ex2(-1.44269504f * z));
}

// y = act(z), s = act'(z).
template <int ACT, bool EXACT>
__device__ __forceinline__ void activate(float z, float &y, float &s)
{
    if constexpr (ACT == SGEMM_ACT_RELU) {
        y = z > 0.0f ? z : z != z ? z : 0.0f;
        s = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    } else if constexpr (ACT == SGEMM_ACT_GELU) {
        float below, density;  // the normal distribution and its density times sqrt(2 pi)
        if constexpr (EXACT) {
            density = expf(-0.5f * z * z);
            below = normcdff(z);
        } else {
            const float a = 0.707106781f * fabsf(z), t = rcp(fmaf(0.495f, a, 1.0f));
            density = ex2(-0.721347520f * z * z);
            const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, -0.193083391f, 0.543523073f), 0.0466414914f), 0.327883065f),
                                     0.275034666f);
            const float tail = 0.5f * q * density;
            below = z >= 0.0f ? 1.0f - tail : tail;
        }
        y = z * below;
        s = fmaf(z * density, 0.398942280f, below);
    } else if constexpr (ACT == SGEMM_ACT_GELU_TANH) {
        const float c = fminf(fmaxf(z, -20.0f), 20.0f);  // beyond it the slope is 0 or 1, and the square may leave FP32
        const float q = sigmoid<EXACT>(1.595769122f * fmaf(0.044715f * c * c, c, c));
        y = z * q;
        s = fmaf(c * q * (1.0f - q), fmaf(0.2140644488f, c * c, 1.595769122f), q);
        if (z != z) s = z;
    } else if constexpr (ACT == SGEMM_ACT_SILU) {
        const float q = sigmoid<EXACT>(z);
        y = z * q;
        s = q * fmaf(z, 1.0f - q, 1.0f);
    } else {
        y = z;
        s = 1.0f;
    }
}

template <bool EXACT>
__device__ __forceinline__ void activate_by(int act, float z, float &y, float &s)
{
    switch (act) {
    case SGEMM_ACT_RELU: activate<SGEMM_ACT_RELU, EXACT>(z, y, s); break;
    case SGEMM_ACT_GELU: activate<SGEMM_ACT_GELU, EXACT>(z, y, s); break;
    case SGEMM_ACT_GELU_TANH: activate<SGEMM_ACT_GELU_TANH, EXACT>(z, y, s); break;
    case SGEMM_ACT_SILU: activate<SGEMM_ACT_SILU, EXACT>(z, y, s); break;
    default: activate<SGEMM_ACT_NONE, EXACT>(z, y, s);
    }
}

// A slope as it is kept beside bfloat16 operands, and back.
constexpr float kSlopeUnit = 1.0f / 16384.0f;

__device__ __forceinline__ short slope_close(float s)
{
    return s != s ? static_cast<short>(-32768) : static_cast<short>(__float2int_rn(s * 16384.0f));
}

__device__ __forceinline__ float slope_open(short s)
{
    return s == -32768 ? __int_as_float(0x7fffffff) : static_cast<float>(s) * kSlopeUnit;
}

}  // namespace sgemm_dev
