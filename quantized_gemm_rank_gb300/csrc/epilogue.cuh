// epilogue.cuh -- the fused epilogues of the 16-bit matrix products, on some
// consecutive columns at a time.  All arithmetic is fp32; each output is rounded once.
#pragma once

#include <type_traits>

#include "num.cuh"

namespace mc2 {

// The form of a product's epilogue, a template argument of its kernels:
//   EPI_PLAIN     out = acc + bias
//   EPI_FORWARD   z = acc + bias (the optional pre-activation output), out = act(z) (+ aux)
//   EPI_BACKWARD  out = acc * act'(aux)
//   EPI_SCALED    z = float(acc) * scale of the row * scale of the column + bias, acc an exact
//                 integer sum of 8-bit codes (held as fp16), out = act(z) (+ aux)
//   EPI_SUMS      acc itself, in 32 bits: a part of a split contraction
enum EpiMode : int { EPI_PLAIN = 0, EPI_FORWARD = 1, EPI_BACKWARD = 2, EPI_SCALED = 3, EPI_SUMS = 4 };

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

// v: z of kN columns (EPI_FORWARD, EPI_SCALED), or the product (EPI_BACKWARD); a: their aux, two
// columns a word.
template <bool kBF16, int kEpi, int kN>
__device__ __forceinline__ void epilogue(float (&v)[kN], const uint32_t (&a)[kN / 2], const Activation &act, bool has_aux) {
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            const float2 r = f(make_float2(v[2 * i], v[2 * i + 1]), unpack2<kBF16>(a[i]));
            v[2 * i] = r.x;
            v[2 * i + 1] = r.y;
        }
    };
    // (one loop for each form: the choice is made once for all kN columns)
    auto apply = [&](auto form) {
        Activation one = act;
        one.form = decltype(form)::value;
        if constexpr (kEpi != EPI_BACKWARD)
            each([&](float2 z, float2) { return act2(z, one); });
        else
            each([&](float2 z, float2 x) { return __fmul2_rn(z, act_derivative2(x, one)); });
    };
    switch (act.form) {
        case CASE_RELU: apply(std::integral_constant<int, CASE_RELU>{}); break;
        case CASE_ERF: apply(std::integral_constant<int, CASE_ERF>{}); break;
        case CASE_SIGMOID: apply(std::integral_constant<int, CASE_SIGMOID>{}); break;
        default: break;
    }
    if (kEpi != EPI_BACKWARD && has_aux) each([](float2 z, float2 x) { return __fadd2_rn(z, x); });
}

}  // namespace mc2
