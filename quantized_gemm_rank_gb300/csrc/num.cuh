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

// An activation as its kernels take it.  silu, z / (1 + e^-z), and the tanh form of
// gelu, z (1 + tanh u) / 2 = z / (1 + e^-2u) with u = sqrt(2/pi) (z + 0.044715 z^3), are one
// function, z sigmoid(z (c1 + c2 z^2)), with (1, 0) and 2 sqrt(2/pi) (1, 0.044715).
enum ActCase : int { CASE_NONE = 0, CASE_RELU = 1, CASE_ERF = 2, CASE_SIGMOID = 3 };
struct Activation {
    int form;        // ActCase
    float c1, c2;    // CASE_SIGMOID
    float limit;     // CASE_SIGMOID: |z| from which the sigmoid is taken to be constant: below 3e-18, or 1
};

inline Activation activation_of(int act) {
    constexpr float kSqrt2OverPi = 0.79788456080286536f;
    switch (act) {
        case ACT_RELU: return {CASE_RELU, 0.0f, 0.0f, 0.0f};
        case ACT_GELU: return {CASE_ERF, 0.0f, 0.0f, 0.0f};
        case ACT_GELU_TANH: return {CASE_SIGMOID, 2.0f * kSqrt2OverPi, 2.0f * kSqrt2OverPi * 0.044715f, 7.4f};
        case ACT_SILU: return {CASE_SIGMOID, 1.0f, 0.0f, 40.5f};
        default: return {CASE_NONE, 0.0f, 0.0f, 0.0f};
    }
}

// The special function unit takes a warp eight cycles an operation and the rest of an
// epilogue little more, so the functions below work on pairs: one reciprocal for both
// (1/a = b r, 1/b = a r with r = 1/(ab)), and packed fp32 arithmetic.
__device__ __forceinline__ float exp2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float2 reciprocals(float2 d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
    return make_float2(r * d.y, r * d.x);
}

// z held inside [lo, hi]; a NaN is kept.
__device__ __forceinline__ float hold(float z, float lo, float hi) {
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(z), "f"(lo));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(c), "f"(hi));
    return c;
}
__device__ __forceinline__ float2 hold2(float2 z, float lo, float hi) { return make_float2(hold(z.x, lo, hi), hold(z.y, lo, hi)); }
// The same where a NaN must not reach a pair's common reciprocal: it becomes lo, and
// comes back by the factor that z itself is.
__device__ __forceinline__ float2 inside2(float2 z, float lo, float hi) {
    return make_float2(fminf(fmaxf(z.x, lo), hi), fminf(fmaxf(z.y, lo), hi));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSqrtHalf = 0.70710678118654752f;     // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1 / sqrt(2 pi)
constexpr float kErfLimit = 14.0f;                    // e^(-14^2 / 2) is below fp32's range

// sigmoid(c (c1 + c2 c^2)) for |c| <= limit, where e^-t of two is within fp32's range
__device__ __forceinline__ float2 sigmoid_form2(float2 c, const Activation &a) {
    const float2 t = __ffma2_rn(__fmul2_rn(c, c), both(-a.c2 * kLog2e), both(-a.c1 * kLog2e));
    const float2 x = __fmul2_rn(c, t);
    return reciprocals(__fadd2_rn(make_float2(exp2_f(x.x), exp2_f(x.y)), both(1.0f)));
}

// The normal distribution at |z| <= kErfLimit: Phi(z) = (1 + erf(z / sqrt 2)) / 2 and, for the
// derivative, e^(-z^2 / 2).  erf by Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26: for x >= 0, erf x = 1 - (a1 t + ... + a5 t^5) e^(-x^2), t = 1 / (1 + p x),
// to 1.5e-7; its exponential is the density's, so the derivative costs little more
// than the value.
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2 &expo) {
    constexpr float kP = 0.3275911f * kSqrtHalf;
    const float2 t = reciprocals(make_float2(fmaf(fabsf(z.x), kP, 1.0f), fmaf(fabsf(z.y), kP, 1.0f)));
    const float2 x = __fmul2_rn(__fmul2_rn(z, z), both(-0.5f * kLog2e));
    expo = make_float2(exp2_f(x.x), exp2_f(x.y));
    float2 q = __ffma2_rn(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
    q = __ffma2_rn(q, t, both(0.5f * 1.421413741f));
    q = __ffma2_rn(q, t, both(0.5f * -0.284496736f));
    q = __ffma2_rn(q, t, both(0.5f * 0.254829592f));
    const float2 tail = __fmul2_rn(__fmul2_rn(q, t), expo);   // Phi(-|z|)
    return make_float2(z.x < 0.0f ? tail.x : 1.0f - tail.x, z.y < 0.0f ? tail.y : 1.0f - tail.y);
}

// act(z).  Far below zero silu and gelu are taken at their limit's argument (their value
// there is below 2e-16), so an infinity gives its limit and not infinity times zero.
__device__ __forceinline__ float2 act2(float2 z, const Activation &a) {
    switch (a.form) {   // the same in every thread
        case CASE_RELU: return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);   // (a NaN stays one)
        case CASE_ERF: {
            float2 e;
            const float2 phi = normal_cdf2(inside2(z, -kErfLimit, kErfLimit), e);
            const float top = __int_as_float(0x7F800000);
            return __fmul2_rn(hold2(z, -kErfLimit, top), phi);
        }
        case CASE_SIGMOID: {
            const float top = __int_as_float(0x7F800000);
            return __fmul2_rn(hold2(z, -a.limit, top), sigmoid_form2(inside2(z, -a.limit, a.limit), a));
        }
        default: return z;
    }
}

// act'(z), for z held where it has not yet reached its limit:
//   relu  1 above 0;  erf form  Phi(z) + z phi(z);  sigmoid form  s + z s (1 - s) (c1 + 3 c2 z^2)
__device__ __forceinline__ float2 act_derivative2(float2 z, const Activation &a) {
    switch (a.form) {
        case CASE_RELU: return make_float2(z.x > 0.0f ? 1.0f : 0.0f, z.y > 0.0f ? 1.0f : 0.0f);
        case CASE_ERF: {
            const float2 c = hold2(z, -kErfLimit, kErfLimit);
            float2 e;
            const float2 phi = normal_cdf2(inside2(z, -kErfLimit, kErfLimit), e);
            return __ffma2_rn(__fmul2_rn(c, both(kInvSqrt2Pi)), e, phi);
        }
        case CASE_SIGMOID: {
            const float2 c = hold2(z, -a.limit, a.limit);
            const float2 s = sigmoid_form2(inside2(z, -a.limit, a.limit), a);
            const float2 slope = __ffma2_rn(__fmul2_rn(c, c), both(3.0f * a.c2), both(a.c1));
            const float2 rest = __fmul2_rn(__fmul2_rn(c, s), __ffma2_rn(s, both(-1.0f), both(1.0f)));
            return __ffma2_rn(rest, slope, s);
        }
        default: return both(1.0f);
    }
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
