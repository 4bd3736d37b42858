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

// Packed pairs of FP32: one instruction for two elements. The epilogues below are bound
// by instruction issue, and most of an activation is multiply-adds.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// max(z, 0) that keeps a NaN.
__device__ __forceinline__ float relu_nan(float z)
{
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
    return y;
}

// max of two magnitudes that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Upper tail of the normal distribution, Q(t) = 1 - Phi(t) at t = |z|, as 2^-p(t):
// log2 Q is smooth, so a polynomial of degree 8 (fitted here to log2 Q on [0, 5.75],
// least maximum error weighted by Q) serves the whole range with one special-function
// operation, where erf takes two branches. |error of Q| < 2.0e-7, |error of t Q| <
// 1.3e-7 (about one FP32 ulp of 1); relative error of Q < 3.4e-5 up to t = 5.5. p keeps
// growing past the fit, so Q goes to 0 from there on (to exactly 0 for an infinite t).
// The argument is s = -|z|, which costs nothing to form and which the callers multiply by.
__device__ __forceinline__ float2 normal_tail2(float2 s)
{
    float2 p = both(-4.72234291e-07f);  // -p, so that 2^ takes it as it is
    p = fma2(p, s, both(-8.03239072e-06f));
    p = fma2(p, s, both(-2.06790246e-05f));
    p = fma2(p, s, both(5.80830500e-04f));
    p = fma2(p, s, both(7.70433247e-03f));
    p = fma2(p, s, both(5.29824905e-02f));
    p = fma2(p, s, both(-4.59033877e-01f));
    p = fma2(p, s, both(1.15112782f));
    p = fma2(p, s, both(-9.99999523e-01f));
    return make_float2(fast_exp2(p.x), fast_exp2(p.y));
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGeluC0 = 0.79788456080286536f;               // sqrt(2 / pi)
constexpr float kGeluC1 = 0.79788456080286536f * 0.044715f;

// act(z) of two elements.
template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 z)
{
    if constexpr (ACT == ACT_RELU) return make_float2(relu_nan(z.x), relu_nan(z.y));
    if constexpr (ACT == ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| Q(|z|), the same on both sides of 0 and
        // without cancellation for z < 0 (the bound keeps an infinite |z| off a zero Q)
        const float2 s = make_float2(fmaxf(-fabsf(z.x), -1.0e4f), fmaxf(-fabsf(z.y), -1.0e4f));
        return fma2(s, normal_tail2(s), make_float2(relu_nan(z.x), relu_nan(z.y)));
    }
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        // z / (1 + 2^w), w = -2 u log2(e) or -z log2(e)
        float2 w;
        if constexpr (ACT == ACT_SILU) w = mul2(z, both(-kLog2e));
        else w = mul2(z, fma2(mul2(z, z), both(-2.0f * kLog2e * kGeluC1), both(-2.0f * kLog2e * kGeluC0)));
        const float2 d = add2(make_float2(fast_exp2(w.x), fast_exp2(w.y)), both(1.0f));
        return mul2(z, make_float2(fast_rcp(d.x), fast_rcp(d.y)));
    }
    return z;
}

// act'(z) of two elements; z finite or NaN (values of a checkpoint).
template <int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z)
{
    if constexpr (ACT == ACT_RELU)
        return make_float2(z.x > 0.0f ? 1.0f : (z.x != z.x ? z.x : 0.0f), z.y > 0.0f ? 1.0f : (z.y != z.y ? z.y : 0.0f));
    if constexpr (ACT == ACT_GELU) {
        // Phi(z) = 1/2 + sign(z) (1/2 - Q(|z|)); a z too large for z^2 meets a density of 0
        const float2 q = normal_tail2(make_float2(-fabsf(z.x), -fabsf(z.y)));
        const float2 e = mul2(mul2(z, z), both(-0.5f * kLog2e));
        const float2 density = mul2(make_float2(fast_exp2(e.x), fast_exp2(e.y)), both(0.398942280401432678f));
        const float2 h = add2(make_float2(-q.x, -q.y), both(0.5f));
        const float2 phi = add2(make_float2(copysignf(h.x, z.x), copysignf(h.y, z.y)), both(0.5f));
        return fma2(z, density, phi);
    }
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        // With e = exp(-|x|) <= 1 and r = 1 / (1 + e), s(x) is r or e r by the sign of x
        // and s (1 - s) = e r^2: nothing overflows or cancels. Past |z| = 100 that product
        // is 0; the clamp keeps its factor finite.
        const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
        const float2 c = make_float2(fmaxf(fminf(z.x, 100.0f), -100.0f), fmaxf(fminf(z.y, 100.0f), -100.0f));
        float2 u, cdu;  // -|x| log2(e), c x'
        if constexpr (ACT == ACT_SILU) {
            u = mul2(a, both(-kLog2e));
            cdu = c;
        } else {
            u = mul2(a, fma2(mul2(z, z), both(-2.0f * kLog2e * kGeluC1), both(-2.0f * kLog2e * kGeluC0)));
            cdu = mul2(c, fma2(mul2(c, c), both(6.0f * kGeluC1), both(2.0f * kGeluC0)));
        }
        const float2 e = make_float2(fast_exp2(u.x), fast_exp2(u.y));
        const float2 d = add2(e, both(1.0f));
        const float2 r = make_float2(fast_rcp(d.x), fast_rcp(d.y));
        const float2 er = mul2(e, r);
        return fma2(cdu, mul2(er, r), make_float2(z.x < 0.0f ? er.x : r.x, z.y < 0.0f ? er.y : r.y));
    }
    return both(1.0f);
}

// act of N values in place.
template <int ACT, int N>
__device__ __forceinline__ void act_values(float *v)
{
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 y = act_value2<ACT>(make_float2(v[e], v[e + 1]));
        v[e] = y.x;
        v[e + 1] = y.y;
    }
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
