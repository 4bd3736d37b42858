// bm_act.cuh -- the activations of an MLP and their derivatives in FP32, and the
// decoding of MXFP8 values (E4M3 codes with one UE8M0 scale per 32 elements).
//
//   relu       max(z, 0)                         [z > 0]
//   gelu       z Phi(z)                          Phi(z) + z phi(z)
//   gelu_tanh  z s, s = 1 / (1 + exp(-2 u)),     s + z s (1 - s) 2 u',
//              u = sqrt(2/pi)(z + 0.044715 z^3)  u' = sqrt(2/pi)(1 + 3 * 0.044715 z^2)
//   silu       z s, s = 1 / (1 + exp(-z))        s + z s (1 - s)
// (gelu_tanh: z (1 + tanh u) / 2 with 1 + tanh u = 2 / (1 + exp(-2 u)).)
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace bm {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// 2^x and 1/x of the special-function unit (about 2 ulp and 1 ulp); ex2 gives +0
// for -inf and inf for +inf.
__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max(z, 0) that keeps a NaN.
__device__ __forceinline__ float relu_nan(float z)
{
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
    return y;
}

// Upper tail of the normal distribution, Q(t) = 1 - Phi(t), for t >= 0, as
// 2^-p(t): log2 Q is smooth, so a polynomial of degree 8 (fitted here to
// log2 Q on [0, 5.75], least maximum error weighted by Q) serves the whole
// range with one special-function operation, where erf takes two branches.
// |error of Q| < 2.0e-7, |error of t Q| < 1.3e-7 (about one FP32 ulp of 1);
// relative error of Q < 3.4e-5 up to t = 5.5. p keeps growing past the fit, so Q
// goes to 0 from there on. t is finite.
__device__ __forceinline__ float normal_tail(float t)
{
    float p = 4.72234291e-07f;
    p = fmaf(p, t, -8.03239072e-06f);
    p = fmaf(p, t, 2.06790246e-05f);
    p = fmaf(p, t, 5.80830500e-04f);
    p = fmaf(p, t, -7.70433247e-03f);
    p = fmaf(p, t, 5.29824905e-02f);
    p = fmaf(p, t, 4.59033877e-01f);
    p = fmaf(p, t, 1.15112782f);
    p = fmaf(p, t, 9.99999523e-01f);
    return fast_exp2(-p);
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGeluC0 = 0.79788456080286536f;               // sqrt(2 / pi)
constexpr float kGeluC1 = 0.79788456080286536f * 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == ACT_RELU) return relu_nan(z);
    if constexpr (ACT == ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| Q(|z|), the same on both sides of 0 and
        // without cancellation for z < 0
        const float t = fminf(fabsf(z), 1.0e4f);
        return fmaf(-t, normal_tail(t), relu_nan(z));
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float w = z * fmaf(-2.0f * kLog2e * kGeluC1, z * z, -2.0f * kLog2e * kGeluC0);  // -2 u log2(e)
        return z * fast_rcp(1.0f + fast_exp2(w));
    }
    if constexpr (ACT == ACT_SILU) return z * fast_rcp(1.0f + fast_exp2(-kLog2e * z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if constexpr (ACT == ACT_GELU) {
        const float t = fminf(fabsf(z), 1.0e4f);
        const float q = normal_tail(t);
        const float density = 0.398942280401432678f * fast_exp2(-0.5f * kLog2e * z * z);
        return fmaf(fmaxf(fminf(z, 1.0e4f), -1.0e4f), density, z >= 0.0f ? 1.0f - q : (z != z ? z : q));
    }
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        // With e = exp(-|x|) <= 1 and r = 1 / (1 + e), s(x) is r or e r by the sign of x
        // and s (1 - s) = e r^2: nothing overflows or cancels. Past |z| = 100 that product
        // is 0; the clamp keeps its factor finite.
        const float c = fmaxf(fminf(z, 100.0f), -100.0f);
        const float u = ACT == ACT_SILU ? fabsf(z) : fabsf(z) * fmaf(2.0f * kGeluC1, z * z, 2.0f * kGeluC0);
        const float du = ACT == ACT_SILU ? 1.0f : fmaf(6.0f * kGeluC1, c * c, 2.0f * kGeluC0);
        const float e = fast_exp2(-kLog2e * u);
        const float r = fast_rcp(1.0f + e);
        return fmaf(c * du, e * r * r, z < 0.0f ? e * r : r);
    }
    return 1.0f;
}

// f(integral_constant<ACT>) for the activation `act`: one switch around a whole
// unrolled block instead of one per element.
template <int A>
struct ActTag {
    static constexpr int value = A;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F &&f)
{
    switch (act) {
    case ACT_RELU: f(ActTag<ACT_RELU>{}); break;
    case ACT_GELU: f(ActTag<ACT_GELU>{}); break;
    case ACT_GELU_TANH: f(ActTag<ACT_GELU_TANH>{}); break;
    case ACT_SILU: f(ActTag<ACT_SILU>{}); break;
    default: f(ActTag<ACT_NONE>{}); break;
    }
}

// ---------------------------------------------------------------- MXFP8 values
// Value of a UE8M0 code: 2^(code - 127); code 0 is a subnormal, 255 NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t code)
{
    return __uint_as_float(code == 0u ? 0x00400000u : (code == 255u ? 0x7FFFFFFFu : code << 23));
}

// Four E4M3 codes (lowest byte first) as FP32.
__device__ __forceinline__ void e4m3x4_values(uint32_t codes, float (&v)[4])
{
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

}  // namespace bm
