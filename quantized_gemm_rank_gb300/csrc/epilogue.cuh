// epilogue.cuh -- the fused epilogues of the 16-bit matrix products, on some
// consecutive columns at a time.  All arithmetic is fp32; each output is rounded once.
#pragma once

#include "num.cuh"

namespace mc2 {

// The form of a product's epilogue, a template argument of its kernels:
//   EPI_PLAIN     out = acc + bias
//   EPI_FORWARD   z = acc + bias (the optional pre-activation output), out = act(z) (+ aux)
//   EPI_BACKWARD  out = acc * act'(aux)
enum EpiMode : int { EPI_PLAIN = 0, EPI_FORWARD = 1, EPI_BACKWARD = 2 };

// An activation as its kernels take it.  silu and the tanh form of gelu are one
// function, z sigmoid(z (c1 + c2 z^2)), with (1, 0) and 2 sqrt(2/pi) (1, 0.044715):
// so the epilogues hold four cases and not five.
enum ActCase : int { CASE_NONE = 0, CASE_RELU = 1, CASE_ERF = 2, CASE_SIGMOID = 3 };
struct Activation {
    int form;        // ActCase
    float c1, c2;    // CASE_SIGMOID
    float limit;     // CASE_SIGMOID: |z| from which the sigmoid is 0 or 1 in fp32
};

inline Activation activation_of(int act) {
    switch (act) {
        case ACT_RELU: return {CASE_RELU, 0.0f, 0.0f, 0.0f};
        case ACT_GELU: return {CASE_ERF, 0.0f, 0.0f, 0.0f};
        case ACT_GELU_TANH: return {CASE_SIGMOID, 2.0f * kSqrt2OverPi, 2.0f * kSqrt2OverPi * kGeluCubic, kTanhLimit};
        case ACT_SILU: return {CASE_SIGMOID, 1.0f, 0.0f, kSiluLimit};
        default: return {CASE_NONE, 0.0f, 0.0f, 0.0f};
    }
}

template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (kBF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&v);
    } else {
        __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&v);
    }
}

template <bool kBF16>
__device__ __forceinline__ float load16(const void *base, int idx) {
    const uint16_t v = reinterpret_cast<const uint16_t *>(base)[idx];
    if constexpr (kBF16) {
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    } else {
        return __half2float(__ushort_as_half(v));
    }
}

// Two 16-bit values of one 32-bit word.
template <bool kBF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (kBF16) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
}

// The biases of columns col .. col + 7, zero from column n on.
template <bool kBF16>
__device__ __forceinline__ void load_bias8(const void *bias, int col, int n, float (&b)[8]) {
    const uint16_t *p = static_cast<const uint16_t *>(bias) + col;
    if (col + 8 <= n && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<kBF16>(w[i]);
            b[2 * i] = f.x;
            b[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = col + i < n ? load16<kBF16>(bias, col + i) : 0.0f;
    }
}

// v: z of kN columns (EPI_FORWARD), or the product (EPI_BACKWARD); a: their aux, two
// columns a word.
template <bool kBF16, int kEpi, int kN>
__device__ __forceinline__ void epilogue(float (&v)[kN], const uint32_t (&a)[kN / 2], const Activation &act, bool has_aux) {
    auto aux = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            const float2 x = unpack2<kBF16>(a[i]);
            f(v[2 * i], x.x);
            f(v[2 * i + 1], x.y);
        }
    };
    if constexpr (kEpi == EPI_FORWARD) {
        switch (act.form) {   // the same in every thread
            case CASE_RELU:
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] = act_f<ACT_RELU>(v[i]);
                break;
            case CASE_ERF:
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] = act_f<ACT_GELU>(v[i]);
                break;
            case CASE_SIGMOID:
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] = sigmoid_form(v[i], act.c1, act.c2, act.limit);
                break;
            default: break;
        }
        if (has_aux) aux([](float &z, float x) { z = __fadd_rn(z, x); });
    } else {
        switch (act.form) {
            case CASE_RELU: aux([](float &z, float x) { z *= act_derivative_f<ACT_RELU>(x); }); break;
            case CASE_ERF: aux([](float &z, float x) { z *= act_derivative_f<ACT_GELU>(x); }); break;
            case CASE_SIGMOID:
                aux([&](float &z, float x) { z *= sigmoid_form_derivative(x, act.c1, act.c2, act.limit); });
                break;
            default: break;
        }
    }
}

}  // namespace mc2
