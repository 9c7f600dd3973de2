// Activations of the dense projections, their slopes, and the arguments of the
// element-wise end of a tile, shared by the CUDA-core and the tensor-core kernels.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "moe.h"

namespace moe {
namespace lin {

// e^(-z^2 / 2) and the normal distribution's Phi(z), fp32.  For x = |z| and
// r = 1 / (x + 3), (x + 3) e^(x^2 / 2) Phi(-x) is smooth in t = 1 - 6 r, which
// runs from -1 at x = 0 to 1; the polynomial is its fit of least relative error
// over 0 <= x <= 14 (5e-8; weighted least squares on values to 40 digits), with
// coefficients that fall off, so little is lost to rounding.  Phi is within 2e-7,
// and below 0 within 1.5e-6 of itself down to -8 (the exponent's rounding grows
// with z^2).  It shares its exponential with the density; a library's error
// function next to an exponential costs twice the instructions, and the
// element-wise GELU gradient is bound by them.
__device__ __forceinline__ void normal_cdf(float z, float &phi, float &e)
{
    e = exp_32(-0.5f * z * z);
    const float r = recip_32(fabsf(z) + 3.0f);
    const float t = fmaf(-6.0f, r, 1.0f);
    float q = fmaf(-2.66765798e-4f, t, -9.03251872e-4f);
    q = fmaf(q, t, 1.07603637e-3f);
    q = fmaf(q, t, 6.92392187e-3f);
    q = fmaf(q, t, -1.04799354e-2f);
    q = fmaf(q, t, -4.72561009e-2f);
    q = fmaf(q, t, 2.30019346e-1f);
    q = fmaf(q, t, -5.09332299e-1f);
    q = fmaf(q, t, 7.29083657e-1f);
    q *= r * e;
    phi = z < 0.0f ? q : 1.0f - q;
}

// z kept between lo and hi, a NaN as it is: outside, the functions below are
// their limits (what is left of them lies below the smallest normal number times
// |z|), and no product meets an infinity.  The reciprocal of 1 + e^88 flushes to 0.
__device__ __forceinline__ float within(float z, float lo, float hi)
{
    return z < lo ? lo : (z > hi ? hi : z);
}

// act(z), fp32.  The tanh form of GELU is z times a logistic function:
// (1 + tanh u) / 2 = 1 / (1 + e^{-2u}).
template <int ACT>
__device__ __forceinline__ float act_fwd(float z)
{
    if (ACT == MOE_LINEAR_RELU)
        return z < 0.0f ? 0.0f : z;      // a NaN stays one
    if (ACT == MOE_LINEAR_SILU) {
        z = z < -88.0f ? -88.0f : z;
        return z * recip_32(1.0f + exp_32(-z));
    }
    if (ACT == MOE_LINEAR_GELU) {
        z = z < -20.0f ? -20.0f : z;
        float phi, e;
        normal_cdf(z, phi, e);
        return z * phi;
    }
    if (ACT == MOE_LINEAR_GELU_TANH) {
        z = z < -20.0f ? -20.0f : z;
        const float u = 0.79788456080286536f * fmaf(0.044715f * z, z * z, z);
        return z * recip_32(1.0f + exp_32(fminf(-2.0f * u, 88.0f)));
    }
    return z;
}

// act'(z), fp32.
template <int ACT>
__device__ __forceinline__ float act_bwd(float z)
{
    if (ACT == MOE_LINEAR_RELU)
        return z > 0.0f ? 1.0f : 0.0f;
    if (ACT == MOE_LINEAR_SILU) {
        z = within(z, -88.0f, 88.0f);
        const float s = recip_32(1.0f + exp_32(-z));
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if (ACT == MOE_LINEAR_GELU) {
        z = within(z, -20.0f, 20.0f);
        float phi, e;
        normal_cdf(z, phi, e);
        return fmaf(z * 0.39894228040143268f, e, phi);
    }
    if (ACT == MOE_LINEAR_GELU_TANH) {
        z = within(z, -20.0f, 20.0f);
        const float u = 0.79788456080286536f * fmaf(0.044715f * z, z * z, z);
        const float p = recip_32(1.0f + exp_32(fminf(-2.0f * u, 88.0f)));
        const float du = 0.79788456080286536f * fmaf(3.0f * 0.044715f * z, z, 1.0f);
        return fmaf(2.0f * z * du, p * (1.0f - p), p);
    }
    return 1.0f;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// What is done to a sum before it is stored; the kernels apply it to the pieces
// of a tile that they hold.
struct Epilogue {
    void *out;               // [rows, ldo]
    int64_t ldo;
    const float *bias;       // [cols] or null
    const void *residual;    // [rows, ldr] of the output type, or null
    int64_t ldr;
    void *preact;            // [rows, cols] of the operand type, or null: sum + bias
    int32_t cols;
};

// Calls f with the activation as a constant.
template <typename F>
void with_act(int act, F f)
{
    switch (act) {
    case MOE_LINEAR_RELU: f(std::integral_constant<int, MOE_LINEAR_RELU>()); break;
    case MOE_LINEAR_SILU: f(std::integral_constant<int, MOE_LINEAR_SILU>()); break;
    case MOE_LINEAR_GELU: f(std::integral_constant<int, MOE_LINEAR_GELU>()); break;
    case MOE_LINEAR_GELU_TANH: f(std::integral_constant<int, MOE_LINEAR_GELU_TANH>()); break;
    default: f(std::integral_constant<int, MOE_LINEAR_NONE>()); break;
    }
}

}  // namespace lin
}  // namespace moe
