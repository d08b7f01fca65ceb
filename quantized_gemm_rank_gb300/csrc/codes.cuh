// codes.cuh -- 16-byte vectors of values and their 8-bit codes, shared by the kernels
// that make codes (the norm, an activation that is kept).
#pragma once

#include "num.cuh"

namespace mc2 {

template <int kT>
struct Vec {
    static constexpr int kW = kT == ELEM_F32 ? 4 : 8;   // elements of 16 bytes
};

template <int kT>
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[Vec<kT>::kW]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kT == ELEM_F32) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (kT == ELEM_BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = h.x;
            f[2 * i + 1] = h.y;
        }
    }
}

template <int kT>
__device__ __forceinline__ uint4 pack(const float (&f)[Vec<kT>::kW]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kT == ELEM_F32) {
            w[i] = __float_as_uint(f[i]);
        } else if constexpr (kT == ELEM_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes that are read once: not kept in L1.
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(reinterpret_cast<uint64_t>(p)));
    return v;
}

// The larger of a and |b|; a NaN is kept.
__device__ __forceinline__ float max_abs(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// Largest value over the block: one barrier, the warps' values in slots of their own.
__device__ __forceinline__ uint32_t block_max32(uint32_t v, uint32_t *slots) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (blockDim.x == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, lane < (blockDim.x >> 5) ? slots[lane] : 0u);
}

// A scale that codes can be made with; the others give zeros.
__device__ __forceinline__ bool usable(float step) { return step > 0.0f && step < __int_as_float(0x7F800000); }

// The quotients y / step of a vector by one reciprocal for all of them and
// Markstein's correction (IBM J. Res. Dev. 34, 1990): with inv the rounded
// reciprocal, r = y inv is corrected by its exact remainder, r + (y - r step) inv.
// The result is the rounded quotient, but for quotients within 2^-46 of the middle
// of two floats, where it may be the other one.  Three operations an element: the
// IEEE division of every element set the kernel's time (4096 x 8192 to int8: 51.7 us
// against 40.9 with this).  The remainder must not underflow, so steps below 2^-80 and
// above 1e30 are divided by; a step that is zero, infinite or a NaN gives zeros.
template <int kN>
__device__ __forceinline__ void quotients(const float (&y)[kN], float step, float (&r)[kN]) {
    if (step > 8.2718061e-25f && step < 1e30f) {
        const float inv = __frcp_rn(step);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float q = __fmul_rn(y[e], inv);
            r[e] = __fmaf_rn(__fmaf_rn(-q, step, y[e]), inv, q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kN; ++e) r[e] = usable(step) ? __fdiv_rn(y[e], step) : 0.0f;
    }
}

// The codes of one vector, in one store.
template <int kN>
__device__ __forceinline__ void store_codes(void *q, int64_t at, const float (&r)[kN], int kind) {
    uint32_t w[kN / 4];
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
        if (kind == Q_I8) {
            // |r| is clamped to 127 and 1.5 * 2^23 added: the sum rounds r to an integer, to
            // nearest-even, whose two's complement is its low byte
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                b[e] = __float_as_uint(fminf(fmaxf(r[4 * i + e], -127.0f), 127.0f) + 12582912.0f);
            w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        } else {
            const __nv_fp8_interpretation_t t = kind == Q_E4M3 ? __NV_E4M3 : __NV_E5M2;
            w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(r[4 * i], r[4 * i + 1]), __NV_SATFINITE, t)) |
                   static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(r[4 * i + 2], r[4 * i + 3]), __NV_SATFINITE, t))
                       << 16;
        }
    }
    if constexpr (kN == 8)
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(q) + at) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(q) + at) = w[0];
}

// 1 / Q, rounded: the scale of an activation that is kept is its largest value times this (one product a group, and
// what a tensor divided by the number Q is in torch on a GPU; the rounded quotient may be the float beside it).
__device__ __forceinline__ float q_inverse(int kind) { return kind == Q_I8 ? 1.0f / 127.0f : (kind == Q_E4M3 ? 1.0f / 448.0f : 1.0f / 57344.0f); }

// ------------------------------------------------------------------ from codes to values
// The value of a code, in units of its scale (exact).
__device__ __forceinline__ float decode8(uint32_t code, int kind) {
    if (kind == Q_I8) return static_cast<float>(static_cast<int8_t>(code));
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), kind == Q_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return __half2float(__half(h));
}

// The value of an e8m0 code: 2^(code - 127), of which 2^-127 is subnormal, and NaN for 0xFF.
__device__ __forceinline__ float mx_value(uint32_t code) {
    return code == 0xFFu ? __int_as_float(0x7FC00000) : __uint_as_float(code == 0 ? 0x00400000u : code << 23);
}

// Eight codes, of two words, to their values.
__device__ __forceinline__ void decode_codes(uint2 w, int kind, float (&v)[8]) {
    const uint32_t words[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (kind == Q_I8) {
            // 0x4B000000 + u is the float 2^23 + u: with u = q + 128 it is 2^23 + 128 too large
            const uint32_t u = words[i] ^ 0x80808080u;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * i + e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 + e)) - 8388736.0f;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float2 f;
                if (kind == Q_E5M2) {   // the upper byte of a half
                    const uint32_t h = __byte_perm(words[i], 0, e ? 0x3424 : 0x1404);
                    f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                } else {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(words[i] >> (16 * e)), __NV_E4M3);
                    f = __half22float2(__half2(h));
                }
                v[4 * i + 2 * e] = f.x, v[4 * i + 2 * e + 1] = f.y;
            }
        }
    }
}

// 16 codes of a row, of which `left` are in it (none: 0 or less); zeros behind them.  In one access where they are whole and
// aligned, otherwise by the aligned words that hold one of them at least.  `again`: they will be read again (kept in L1).
__device__ __forceinline__ uint4 load_codes16(const int8_t *from, int left, bool again = false) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(from);
    if (left >= 16 && (a & 15) == 0) return again ? *reinterpret_cast<const uint4 *>(from) : load_once(from);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a & ~uintptr_t(3));
    const int skip = static_cast<int>(a & 3), end = left > 0 ? min(left, 16) + skip : 0;   // in bytes from w on
    uint32_t word[5], q[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) word[i] = 4 * i < end ? w[i] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = __funnelshift_r(word[i], word[i + 1], skip * 8);
        if (left < 4 * i + 4) q[i] = left > 4 * i ? q[i] & ((1u << (8 * (left - 4 * i))) - 1u) : 0;
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

// Columns of a group that share a scale.
__host__ __device__ __forceinline__ int group_size(int qmode) { return qmode == QM_MX ? 32 : 128; }

// The scale of column j of a row of h codes.
template <int kQM>
__device__ __forceinline__ float scale_at(const void *scale, int64_t row, int h, int j) {
    if constexpr (kQM == QM_TOKEN) return static_cast<const float *>(scale)[row];
    if constexpr (kQM == QM_GROUP) return static_cast<const float *>(scale)[row * ((h + 127) / 128) + j / 128];
    return mx_value(static_cast<const uint8_t *>(scale)[row * ((h + 31) / 32) + j / 32]);
}

}  // namespace mc2
