// num.cuh -- device-side number formats and activations shared by the norm and
// the fused-epilogue kernels: loads and stores of fp16/bf16/fp32 values, the
// 8-bit encoders, the activations and their derivatives.  All arithmetic is
// fp32; a value is rounded once, when it is stored.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace mc2 {

// element types, as template arguments
enum ElemKind : int { ELEM_F16 = 0, ELEM_BF16 = 1, ELEM_F32 = 2 };

template <int kT>
struct Elem;
template <>
struct Elem<ELEM_F16> {
    using type = __half;
    static __device__ __forceinline__ float load(const __half *p) { return __half2float(*p); }
    static __device__ __forceinline__ void store(__half *p, float v) { *p = __float2half_rn(v); }
};
template <>
struct Elem<ELEM_BF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
};
template <>
struct Elem<ELEM_F32> {
    using type = float;
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
};

// ------------------------------------------------------------------ activations
enum ActKind : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// 1 / (1 + e^-t).  e^-t overflows to infinity below t = -88 and the quotient is
// then 0, its limit.
__device__ __forceinline__ float sigmoid_f(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

constexpr float kSqrtHalf = 0.70710678118654752f;     // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kTanhLimit = 14.0f;    // e^-2u(14) = e^-218 and e^104 are beyond fp32's range
constexpr float kSiluLimit = 104.0f;

// z sigmoid(t) with t = z (c1 + c2 z^2).  The sigmoid is 0 or 1 in fp32 from |z| =
// limit on, and is taken at z clamped to that, which keeps t finite (0 times
// infinity otherwise); a NaN passes the comparisons unchanged.
__device__ __forceinline__ float sigmoid_form(float z, float c1, float c2, float limit) {
    const float c = z > limit ? limit : (z < -limit ? -limit : z);
    return z * sigmoid_f(c * fmaf(c2, c * c, c1));
}

// Its derivative, s + z s (1 - s) t'(z), at the same clamped z (see below).
__device__ __forceinline__ float sigmoid_form_derivative(float z, float c1, float c2, float limit) {
    const float c = z > limit ? limit : (z < -limit ? -limit : z);
    const float zz = c * c;
    const float s = sigmoid_f(c * fmaf(c2, zz, c1));
    return fmaf(c * s * (1.0f - s), fmaf(3.0f * c2, zz, c1), s);
}

// The normal distribution at z: Phi(z) = (1 + erf(z / sqrt 2)) / 2 and, for the
// derivative, e^(-z^2 / 2).  erf by Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26: for x >= 0, erf x = 1 - (a1 t + ... + a5 t^5) e^(-x^2), t = 1 / (1 + p x),
// to 1.5e-7; its exponential is the density's, so the derivative costs little more
// than the value.  Infinities give the limits (e^-inf = 0, t = 0), a NaN stays one.
__device__ __forceinline__ float normal_cdf(float z, float &expo) {
    const float x = fabsf(z) * kSqrtHalf;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    expo = __expf(-x * x);
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * q * t * expo;   // Phi(-|z|)
    return z < 0.0f ? tail : 1.0f - tail;
}

// relu  max(z, 0) (a NaN stays a NaN)
// gelu  z (1 + erf(z / sqrt 2)) / 2
// gelu_tanh  z (1 + tanh u) / 2 with u = sqrt(2/pi) (z + 0.044715 z^3); as
//       (1 + tanh u) / 2 = 1 / (1 + e^-2u) it is z sigmoid(2u)
// silu  z sigmoid(z)
template <int kAct>
__device__ __forceinline__ float act_f(float z) {
    if constexpr (kAct == ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (kAct == ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if constexpr (kAct == ACT_GELU_TANH)
        return sigmoid_form(z, 2.0f * kSqrt2OverPi, 2.0f * kSqrt2OverPi * kGeluCubic, kTanhLimit);
    if constexpr (kAct == ACT_SILU) return sigmoid_form(z, 1.0f, 0.0f, kSiluLimit);
    return z;
}

// The derivatives.  Each is evaluated at z clamped to a range outside which it
// has reached its limit (0 or 1) in fp32, so that large and infinite z give the
// limit and not infinity times zero; a NaN passes the comparisons unchanged.
template <int kAct>
__device__ __forceinline__ float act_derivative_f(float z) {
    if constexpr (kAct == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (kAct == ACT_GELU) {
        // Phi(z) + z phi(z)
        const float c = z > 14.0f ? 14.0f : (z < -14.0f ? -14.0f : z);
        float e;
        const float cdf = normal_cdf(c, e);
        return fmaf(c * kInvSqrt2Pi, e, cdf);
    }
    if constexpr (kAct == ACT_GELU_TANH)
        return sigmoid_form_derivative(z, 2.0f * kSqrt2OverPi, 2.0f * kSqrt2OverPi * kGeluCubic, kTanhLimit);
    if constexpr (kAct == ACT_SILU) return sigmoid_form_derivative(z, 1.0f, 0.0f, kSiluLimit);
    return 1.0f;
}

// ------------------------------------------------------------------ 8-bit codes
enum QKind : int { Q_I8 = 0, Q_E4M3 = 1, Q_E5M2 = 2 };
enum QMode : int { QM_NONE = 0, QM_TOKEN = 1, QM_GROUP = 2, QM_MX = 3 };

__host__ __device__ __forceinline__ float q_max(int kind) { return kind == Q_I8 ? 127.0f : (kind == Q_E4M3 ? 448.0f : 57344.0f); }
// exponent of the largest power of two the type holds
__host__ __device__ __forceinline__ int q_emax(int kind) { return kind == Q_E4M3 ? 8 : 15; }

// The larger of two absolute values given as bit patterns: as unsigned integers
// they order like the values, with every NaN above infinity, so a NaN is kept.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// A scaled value to its code: ties to even, saturated at the largest finite value.
__device__ __forceinline__ uint32_t encode8(float r, int kind) {
    if (kind == Q_I8) return static_cast<uint32_t>(min(max(__float2int_rn(r), -127), 127)) & 0xFFu;
    return __nv_cvt_float_to_fp8(r, __NV_SATFINITE, kind == Q_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

// mx scale of a group whose largest absolute value has the bits `amax`:
// the code of 2^(floor(log2 amax) - emax), at least 2^-127 (code 0); a group that
// holds an infinity or a NaN gets the NaN code.
__device__ __forceinline__ uint32_t mx_code(uint32_t amax, int kind) {
    if (amax >= 0x7F800000u) return 0xFFu;
    return static_cast<uint32_t>(max(static_cast<int>(amax >> 23) - q_emax(kind), 0));
}
// 2^-(code - 127), the factor from a value to its code's value (codes of finite groups)
__device__ __forceinline__ float mx_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }

}  // namespace mc2
