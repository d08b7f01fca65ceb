// kept_kernels.cu -- an activation kept in 8 bits, and what is made of it.
//
//   y = act(z),  scale = max|y| (1 / Q) over a row or a group,  q = y / scale to nearest-even    (act_quant)
//   out = act(q scale)                                                                           (act_dequant)
//   dz = dy act'(q scale)                                                                        (act_grad_quant)
// Arithmetic is fp32; codes and outputs are rounded once.  Memory bounds all of them without an activation, issue with gelu:
// each element is read once, eight at a time (16 bytes of a 16-bit matrix, 8 of codes).  8192 x 8192 bf16, us (TB/s): to int8 per token
// 36.5 (5.5), with gelu 51, per 128 columns 41.4 (4.9), with gelu 62; from int8 per 128 to 16 bits 35 (5.7), with gelu 47.5;
// gelu' through it 62 (5.4).  fp32 to int8 per token 50 (6.7), per 128 columns 55.5; from int8 per 128 to fp32 75 (4.5), with silu 84,
// with gelu 143: an output of 32 bits is made with CUDA's own functions.
#include "kept.h"

#include "codes.cuh"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 8;      // elements a thread takes at a time
// Blocks an SM holds and rows of a thread on their way at once, of the covering kernels.  8192 x 8192, in us: from codes to 16 bits
// 35 with (8, 1), 38 (6, 1), 37.5 (4, 2); the gradient 62 with (6, 1), 64 (5, 1), 69 (4, 2), 106 (8, 1: registers spill); to codes
// per 128 without an activation and with gelu 44 and 62 with (4, 2), 43.5 and 67 (6, 1), 42 and 64 (4, 3), 46 and 62.5 (3, 3),
// all of them by floats (below).
constexpr int kToBlocks = 4, kToRows = 2, kFromBlocks = 8, kGradBlocks = 6;

// f(activation with its form a constant): the choice is made once for all of a thread's elements.
template <class F>
__device__ __forceinline__ void with_form(const Activation &act, F f) {
    Activation one = act;
    switch (act.form) {   // the same in every thread
        case CASE_RELU: one.form = CASE_RELU; f(one); break;
        case CASE_ERF: one.form = CASE_ERF; f(one); break;
        case CASE_SIGMOID: one.form = CASE_SIGMOID; f(one); break;
        default: one.form = CASE_NONE; f(one); break;
    }
}

// gelu by the tail T = Phi(-|z|) alone: z Phi(z) = max(z, 0) - |z| T, and Phi(z) + z phi(z) is u = |z| phi(z) - T above 1, or
// -u below zero.  Two thirds of the instructions of act2, which selects T or 1 - T (8192 x 8192 bf16 to int8 per 128 69 us, so
// 62; back 52.5 and 47.5), and eight registers fewer than act_derivative2 (65 and 62).  |z| is held where T is 0, so that an
// infinity gives its limit; a NaN is kept out of the pair's common reciprocal and comes back by a factor.
__device__ __forceinline__ float2 held_abs2(float2 z) { return make_float2(fminf(fabsf(z.x), kErfLimit), fminf(fabsf(z.y), kErfLimit)); }

__device__ __forceinline__ float2 gelu2(float2 z) {
    const float2 a = held_abs2(z);
    float2 expo, top;
    const float2 tail = normal_tail2(a, reciprocals(__ffma2_rn(a, both(kErfP), both(1.0f))), expo);
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top.x) : "f"(z.x));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top.y) : "f"(z.y));
    return __ffma2_rn(make_float2(-a.x, -a.y), tail, top);
}

__device__ __forceinline__ float2 gelu_derivative2(float2 z) {
    const float2 a = held_abs2(z);
    float2 expo, c;
    const float2 tail = normal_tail2(a, reciprocals(__ffma2_rn(a, both(kErfP), both(1.0f))), expo);
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(c.x) : "f"(fabsf(z.x)), "f"(kErfLimit));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(c.y) : "f"(fabsf(z.y)), "f"(kErfLimit));
    const float2 u = __ffma2_rn(__fmul2_rn(c, both(kInvSqrt2Pi)), expo, make_float2(-tail.x, -tail.y));
    return make_float2(z.x < 0.0f ? -u.x : 1.0f + u.x, z.y < 0.0f ? -u.y : 1.0f + u.y);
}

__device__ __forceinline__ float2 act_of(float2 z, const Activation &act) { return act.form == CASE_ERF ? gelu2(z) : act2(z, act); }
__device__ __forceinline__ float2 derivative_of(float2 z, const Activation &act) {
    return act.form == CASE_ERF ? gelu_derivative2(z) : act_derivative2(z, act);
}

// The same for an output of 32 bits, by CUDA's own functions: erf's absolute 1.5e-7 above is 5e-4 of gelu(-4) and 1% of gelu(-8), the
// rounded argument of 2^x above 2e-6 of silu(-40) (8192 x 8192 with gelu 143 us, with those 68).  z is held where the value is below
// fp32's range.
__device__ __forceinline__ float act32(float z, const Activation &act) {
    constexpr float kLeast = -104.0f;   // e^-104 is below fp32's range
    const float c = hold(z, act.form == CASE_ERF ? -kErfLimit - 1.0f : kLeast, __int_as_float(0x7F800000));
    if (act.form == CASE_ERF) return c * normcdff(c);
    const float w = fminf(c, -kLeast), e = expf(-fabsf(w * fmaf(w * w, act.c2, act.c1)));
    return c * ((w < 0.0f ? e : 1.0f) / (1.0f + e));
}
template <int kT>
__device__ __forceinline__ float2 value_of(float2 z, const Activation &act) {
    if (kT == ELEM_F32 && (act.form == CASE_ERF || act.form == CASE_SIGMOID)) return make_float2(act32(z.x, act), act32(z.y, act));
    return act_of(z, act);
}

// kT: the type of what becomes of it
template <int kT>
__device__ __forceinline__ void apply_act(float (&y)[kChunk], const Activation &act) {
    with_form(act, [&](const Activation &one) {
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) {
            const float2 v = value_of<kT>(make_float2(y[e], y[e + 1]), one);
            y[e] = v.x, y[e + 1] = v.y;
        }
    });
}

__device__ __forceinline__ void times_derivative(float (&d)[kChunk], const float (&z)[kChunk], const Activation &act) {
    with_form(act, [&](const Activation &one) {
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) {
            const float2 v = __fmul2_rn(make_float2(d[e], d[e + 1]), derivative_of(make_float2(z[e], z[e + 1]), one));
            d[e] = v.x, d[e + 1] = v.y;
        }
    });
}

// Eight elements, as the 16-byte words they are in memory.
template <int kT>
struct Raw {
    uint4 v[kT == ELEM_F32 ? 2 : 1];
};

template <int kT>
__device__ __forceinline__ Raw<kT> load_raw(const void *p) {
    Raw<kT> r;
    r.v[0] = load_once(p);
    if constexpr (kT == ELEM_F32) r.v[1] = load_once(static_cast<const char *>(p) + 16);
    return r;
}

template <int kT>
__device__ __forceinline__ void values(const Raw<kT> &r, float (&f)[kChunk]) {
    if constexpr (kT == ELEM_F32) {
        float a[4], b[4];
        unpack<kT>(r.v[0], a);
        unpack<kT>(r.v[1], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    } else {
        unpack<kT>(r.v[0], f);
    }
}

template <int kT>
__device__ __forceinline__ void store_values(void *p, const float (&f)[kChunk]) {
    uint4 *to = static_cast<uint4 *>(p);
    if constexpr (kT == ELEM_F32) {
        const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
        to[0] = pack<kT>(a), to[1] = pack<kT>(b);
    } else {
        to[0] = pack<kT>(f);
    }
}

__device__ __forceinline__ uint2 load_codes(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(reinterpret_cast<uint64_t>(p)));
    return v;
}

// How a launch covers a matrix: a thread keeps one chunk of columns and goes down the rows; a row takes `lanes` threads of
// a block (a power of two), a block kThreads / lanes rows at a time.
struct Cover {
    int lanes_log2;
    int chunks;   // of a row
};

// ------------------------------------------------------------------ from codes
// Rows of whole chunks: every access is a whole one.
template <int kT, bool kGrad, int kQM>
__global__ void __launch_bounds__(kThreads, kGrad ? kGradBlocks : kFromBlocks) from_kept_kernel(const void *dy, int64_t lddy, const __grid_constant__ Kept p, Activation act,
                                                             void *out, int64_t ldo, Cover cover) {
    constexpr int kE = kT == ELEM_F32 ? 4 : 2;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int lanes = 1 << cover.lanes_log2, per_block = kThreads >> cover.lanes_log2;
    const int c = blockIdx.x * lanes + (threadIdx.x & (lanes - 1));
    if (c >= cover.chunks) return;
    const int j = c * kChunk;
    const int64_t step = static_cast<int64_t>(gridDim.y) * per_block;
    for (int64_t r = static_cast<int64_t>(blockIdx.y) * per_block + (threadIdx.x >> cover.lanes_log2); r < p.m; r += step) {
        const uint2 q = load_codes(static_cast<const uint8_t *>(p.q) + r * p.h + j);
        Raw<kT> d;
        if constexpr (kGrad) d = load_raw<kT>(static_cast<const char *>(dy) + (r * lddy + j) * kE);
        const float scale = scale_at<kQM>(p.scale, r, p.h, j);
        float z[kChunk];
        decode_codes(q, p.qkind, z);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) z[e] = __fmul_rn(z[e], scale);
        char *to = static_cast<char *>(out) + (r * ldo + j) * kE;
        if constexpr (kGrad) {
            float g[kChunk];
            values<kT>(d, g);
            times_derivative(g, z, act);
            store_values<kT>(to, g);
        } else {
            apply_act<kT>(z, act);
            store_values<kT>(to, z);
        }
    }
}

// Eight bytes from any address, by the aligned words that hold them.
__device__ __forceinline__ uint2 load_bytes8(const uint8_t *p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a & ~uintptr_t(3));
    const uint32_t shift = static_cast<uint32_t>(a & 3) * 8;
    const uint32_t w0 = w[0], w1 = w[1];
    if (shift == 0) return make_uint2(w0, w1);
    const uint32_t w2 = w[2];
    return make_uint2(__funnelshift_r(w0, w1, shift), __funnelshift_r(w1, w2, shift));
}

// Rows of any width and alignment: the chunks are those of the output's aligned 16-byte units, the first and the
// last of a row partial; codes and dy come from any address.
template <int kT, bool kGrad, int kQM>
__global__ void __launch_bounds__(kThreads, kGrad ? 4 : 6) from_kept_any_kernel(const void *dy, int64_t lddy, const __grid_constant__ Kept p,
                                                                                Activation act, void *out, int64_t ldo, Cover cover) {
    using E = Elem<kT>;
    using T = typename E::type;
    constexpr int kE = kT == ELEM_F32 ? 4 : 2;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int lanes = 1 << cover.lanes_log2, per_block = kThreads >> cover.lanes_log2;
    const int c = blockIdx.x * lanes + (threadIdx.x & (lanes - 1));
    const int64_t step = static_cast<int64_t>(gridDim.y) * per_block;
    for (int64_t r = static_cast<int64_t>(blockIdx.y) * per_block + (threadIdx.x >> cover.lanes_log2); r < p.m; r += step) {
        T *to = static_cast<T *>(out) + r * ldo;
        const T *from = kGrad ? static_cast<const T *>(dy) + r * lddy : nullptr;
        const uint8_t *q = static_cast<const uint8_t *>(p.q) + r * p.h;
        const int j0 = c * kChunk - static_cast<int>(reinterpret_cast<uintptr_t>(to) / kE % kChunk);
        if (j0 >= 0 && j0 + kChunk <= p.h) {
            float z[kChunk], g[kChunk];
            const uint2 codes = load_bytes8(q + j0);
            Raw<kT> d;
            if constexpr (kGrad) d.v[0] = load_codes16(reinterpret_cast<const int8_t *>(from + j0), 16);
            const float scale = scale_at<kQM>(p.scale, r, p.h, j0);
            decode_codes(codes, p.qkind, z);
            const int border = kQM == QM_TOKEN ? p.h : (j0 / group_size(kQM) + 1) * group_size(kQM);
            if (border >= j0 + kChunk) {
#pragma unroll
                for (int e = 0; e < kChunk; ++e) z[e] = __fmul_rn(z[e], scale);
            } else {   // a chunk reaches into two groups at most
                const float next = scale_at<kQM>(p.scale, r, p.h, border);
#pragma unroll
                for (int e = 0; e < kChunk; ++e) z[e] = __fmul_rn(z[e], j0 + e < border ? scale : next);
            }
            if constexpr (kGrad) {
                values<kT>(d, g);
                times_derivative(g, z, act);
                store_values<kT>(to + j0, g);
            } else {
                apply_act<kT>(z, act);
                store_values<kT>(to + j0, z);
            }
        } else {
            // (elements are paired with themselves: an activation works on pairs)
            for (int j = max(j0, 0); j < min(j0 + kChunk, p.h); ++j) {
                const float z = __fmul_rn(decode8(q[j], p.qkind), scale_at<kQM>(p.scale, r, p.h, j));
                E::store(to + j, kGrad ? E::load(from + j) * derivative_of(both(z), act).x : value_of<kT>(both(z), act).x);
            }
        }
    }
}

// ------------------------------------------------------------------ to codes
// The codes of a thread's chunk, y / step to nearest-even, in one store.  The quotients are those of quotients() in codes.cuh,
// two at a time; |y| is at most the value that the step was made from, so that they need no clamp but where the step lost
// bits to fp32's lower end (there, as at steps that are zero or not finite, quotients() takes over).
__device__ __forceinline__ void store_quotients(void *q, int64_t at, const float (&y)[kChunk], float step, int kind) {
    if (step > 8.2718061e-25f && step < 1e30f) {
        const float2 inv = both(__frcp_rn(step)), minus = both(-step);
        float2 r[kChunk / 2];
#pragma unroll
        for (int e = 0; e < kChunk / 2; ++e) {
            const float2 v = make_float2(y[2 * e], y[2 * e + 1]);
            const float2 t = __fmul2_rn(v, inv);
            r[e] = __ffma2_rn(__ffma2_rn(t, minus, v), inv, t);
        }
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (kind == Q_I8) {   // (as in store_codes)
                const float2 a = __fadd2_rn(r[2 * i], both(12582912.0f)), b = __fadd2_rn(r[2 * i + 1], both(12582912.0f));
                w[i] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                                   __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
            } else {
                const __nv_fp8_interpretation_t t = kind == Q_E4M3 ? __NV_E4M3 : __NV_E5M2;
                w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(r[2 * i], __NV_SATFINITE, t)) |
                       static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(r[2 * i + 1], __NV_SATFINITE, t)) << 16;
            }
        }
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(q) + at) = make_uint2(w[0], w[1]);
    } else {
        float r[kChunk];
        quotients(y, step, r);
        store_codes(q, at, r, kind);
    }
}

// The scale of a group and the codes of a thread's chunk of it, from the group's largest value (as bits).
template <int kQM>
__device__ __forceinline__ void encode_chunk(const Kept &p, const float (&y)[kChunk], uint32_t top, int64_t scale_index, bool writes_scale,
                                             int64_t at) {
    if constexpr (kQM == QM_MX) {
        const uint32_t code = mx_code(top, p.qkind);
        if (writes_scale) static_cast<uint8_t *>(p.scale)[scale_index] = static_cast<uint8_t>(code);
        const float inverse = mx_inverse(code);
        float r[kChunk];
#pragma unroll
        for (int e = 0; e < kChunk; ++e) r[e] = code != 0xFFu ? y[e] * inverse : 0.0f;
        store_codes(p.q, at, r, p.qkind);
    } else {
        const float step = __fmul_rn(__uint_as_float(top), q_inverse(p.qkind));
        if (writes_scale) static_cast<float *>(p.scale)[scale_index] = step;
        store_quotients(p.q, at, y, step, p.qkind);
    }
}

__device__ __forceinline__ uint32_t largest_of(const float (&y)[kChunk]) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) top = max_abs(top, y[e]);
    return __float_as_uint(top);   // of non-negative values: ordered like them
}

// Rows of whole chunks with scales of groups (16 or 4 neighbouring threads), or with one scale a row of at most 32
// chunks (`lanes` threads): covered like from_kept_kernel.
template <int kT, int kQM>
__global__ void __launch_bounds__(kThreads, kToBlocks) act_quant_kernel(const void *z, int64_t ldz, const __grid_constant__ Kept p, Activation act, Cover cover) {
    constexpr int kE = kT == ELEM_F32 ? 4 : 2;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int lanes = 1 << cover.lanes_log2, per_block = kThreads >> cover.lanes_log2;
    const int c = blockIdx.x * lanes + (threadIdx.x & (lanes - 1));
    const bool live = c < cover.chunks;
    const int j = c * kChunk;
    const int group = kQM == QM_TOKEN ? lanes : group_size(kQM) / kChunk;   // threads that share a scale
    const int groups = kQM == QM_TOKEN ? 1 : (p.h + group_size(kQM) - 1) / group_size(kQM);
    const int64_t step = static_cast<int64_t>(gridDim.y) * per_block;
    // (all threads of a block take as many turns, so that the groups' exchanges are whole)
    for (int64_t first = static_cast<int64_t>(blockIdx.y) * per_block; first < p.m; first += kToRows * step) {
        const int64_t r0 = first + (threadIdx.x >> cover.lanes_log2);
        Raw<kT> raw[kToRows];
#pragma unroll
        for (int i = 0; i < kToRows; ++i) {
            const int64_t r = r0 + i * step;
            if (live && r < p.m) raw[i] = load_raw<kT>(static_cast<const char *>(z) + (r * ldz + j) * kE);
        }
        if constexpr (kT != ELEM_F32) {
            static_assert(kToRows == 2, "a word holds the largest values of two rows");
            if (act.form == CASE_NONE) {
                // the largest values as 16-bit patterns without their sign (ordered like the values, a NaN above all), both
                // rows' in one word (8192 x 8192 to int8 per 128 41.4 us, by floats 43.8; mx 39 and 42)
                uint32_t m[kToRows] = {};
#pragma unroll
                for (int i = 0; i < kToRows; ++i) {
                    if (!live || r0 + i * step >= p.m) continue;
                    const uint4 v = raw[i].v[0];
                    m[i] = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
                }
                uint32_t both_tops = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
                for (int o = group / 2; o > 0; o >>= 1) both_tops = __vmaxu2(both_tops, __shfl_xor_sync(0xFFFFFFFFu, both_tops, o));
                float2 tops;
                if constexpr (kT == ELEM_BF16)
                    tops = make_float2(__uint_as_float(both_tops << 16), __uint_as_float(both_tops & 0xFFFF0000u));
                else
                    tops = __half22float2(*reinterpret_cast<const __half2 *>(&both_tops));
#pragma unroll
                for (int i = 0; i < kToRows; ++i) {
                    const int64_t r = r0 + i * step;
                    if (!live || r >= p.m) continue;
                    float y[kChunk];
                    values<kT>(raw[i], y);
                    encode_chunk<kQM>(p, y, __float_as_uint(i ? tops.y : tops.x), r * groups + (kQM == QM_TOKEN ? 0 : c / group),
                                      (threadIdx.x & (group - 1)) == 0, r * p.h + j);
                }
                continue;
            }
        }
#pragma unroll
        for (int i = 0; i < kToRows; ++i) {
            const int64_t r = r0 + i * step;
            const bool here = live && r < p.m;
            float y[kChunk];
            if (here) {
                values<kT>(raw[i], y);
                apply_act<ELEM_BF16>(y, act);   // (codes have fewer bits)
            } else {
#pragma unroll
                for (int e = 0; e < kChunk; ++e) y[e] = 0.0f;
            }
            uint32_t top = largest_of(y);
            for (int o = group / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            if (here) {
                encode_chunk<kQM>(p, y, top, r * groups + (kQM == QM_TOKEN ? 0 : c / group), (threadIdx.x & (group - 1)) == 0, r * p.h + j);
            }
        }
    }
}

// One scale a row, rows of whole chunks: V chunks a thread, kept between the row's largest value and its codes.  One row a
// block, or (kWarpRow) one a warp.
template <int kT, int V, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? kThreads : 1024) act_quant_row_kernel(const void *z, int64_t ldz, const __grid_constant__ Kept p, Activation act) {
    constexpr int kE = kT == ELEM_F32 ? 4 : 2;
    __shared__ uint32_t slots[32];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarpRow && row >= p.m) return;
    const int T = kWarpRow ? 32 : blockDim.x, mine = kWarpRow ? threadIdx.x & 31 : threadIdx.x, chunks = p.h / kChunk;
    const char *from = static_cast<const char *>(z) + row * ldz * kE;
    Raw<kT> raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = mine + i * T;
        if (c < chunks) raw[i] = load_raw<kT>(from + static_cast<int64_t>(c) * (kChunk * kE));
    }
    float y[V][kChunk];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (mine + i * T < chunks) {
            values<kT>(raw[i], y[i]);
            apply_act<ELEM_BF16>(y[i], act);   // (codes have fewer bits)
            top = max(top, largest_of(y[i]));
        }
    }
    top = kWarpRow ? __reduce_max_sync(0xFFFFFFFFu, top) : block_max32(top, slots);
    const float step = __fmul_rn(__uint_as_float(top), q_inverse(p.qkind));
    if (mine == 0) static_cast<float *>(p.scale)[row] = step;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = mine + i * T;
        if (c < chunks) store_quotients(p.q, row * p.h + static_cast<int64_t>(c) * kChunk, y[i], step, p.qkind);
    }
}

// Any sizes, strides and alignments, element by element: a warp takes 128 of a row at a time (one group, or four of mx), lane l
// elements l, l + 32, l + 64 and l + 96.  One scale a row: the row is read twice, by a warp, or (kBlockRow) by a block.
template <int kT, int kQM, bool kBlockRow>
__global__ void __launch_bounds__(kThreads) act_quant_any_kernel(const void *z, int64_t ldz, const __grid_constant__ Kept p, Activation act) {
    using T = typename Elem<kT>::type;
    __shared__ uint32_t slots[32];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = (p.h + 127) / 128;   // of a row
    const auto load = [&](const T *from, int block, float (&y)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = block * 128 + 32 * i + lane;
            y[i] = j < p.h ? Elem<kT>::load(from + j) : 0.0f;
        }
        with_form(act, [&](const Activation &one) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float2 v = act_of(make_float2(y[i], y[i + 1]), one);
                y[i] = v.x, y[i + 1] = v.y;
            }
        });
    };
    const auto largest = [](const float (&y)[4]) {
        return __float_as_uint(max_abs(max_abs(max_abs(max_abs(0.0f, y[0]), y[1]), y[2]), y[3]));
    };
    const auto store = [&](int64_t row, int block, const float (&r)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = block * 128 + 32 * i + lane;
            if (j < p.h) static_cast<uint8_t *>(p.q)[row * p.h + j] = static_cast<uint8_t>(encode8(r[i], p.qkind));
        }
    };
    float y[4], r[4];
    if constexpr (kQM == QM_TOKEN) {
        const int64_t row = kBlockRow ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWarps + warp;
        const int first = kBlockRow ? warp : 0, step = kBlockRow ? kWarps : 1;
        if (!kBlockRow && row >= p.m) return;
        const T *from = static_cast<const T *>(z) + row * ldz;
        uint32_t top = 0;
        for (int b = first; b < blocks; b += step) {
            load(from, b, y);
            top = max(top, largest(y));
        }
        top = kBlockRow ? block_max32(top, slots) : __reduce_max_sync(0xFFFFFFFFu, top);
        const float scale = __fmul_rn(__uint_as_float(top), q_inverse(p.qkind));
        if (lane == 0 && first == 0) static_cast<float *>(p.scale)[row] = scale;
        for (int b = first; b < blocks; b += step) {
            load(from, b, y);
            quotients(y, scale, r);
            store(row, b, r);
        }
    } else {
        const int64_t total = p.m * blocks, step = static_cast<int64_t>(gridDim.x) * kWarps;
        const int groups = (p.h + group_size(kQM) - 1) / group_size(kQM);
        for (int64_t e = static_cast<int64_t>(blockIdx.x) * kWarps + warp; e < total; e += step) {
            const int64_t row = e / blocks;
            const int b = static_cast<int>(e - row * blocks);
            load(static_cast<const T *>(z) + row * ldz, b, y);
            if constexpr (kQM == QM_GROUP) {
                const float scale = __fmul_rn(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, largest(y))), q_inverse(p.qkind));
                if (lane == 0) static_cast<float *>(p.scale)[row * groups + b] = scale;
                quotients(y, scale, r);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t code = mx_code(__reduce_max_sync(0xFFFFFFFFu, abs_bits(y[i])), p.qkind);
                    if (lane == 0 && b * 4 + i < groups) static_cast<uint8_t *>(p.scale)[row * groups + b * 4 + i] = static_cast<uint8_t>(code);
                    r[i] = code != 0xFFu ? y[i] * mx_inverse(code) : 0.0f;
                }
            }
            store(row, b, r);
        }
    }
}

template <class... P, class... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int block, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The cover of rows of `chunks` chunks, at least `least` threads a row, and the grid for it: as many blocks as the device
// holds, of `resident` an SM, each with several rows where there are more.
dim3 cover_rows(int chunks, int least, int64_t m, int num_sms, int resident, Cover *cover) {
    cover->chunks = chunks;
    cover->lanes_log2 = 0;
    while ((1 << cover->lanes_log2) < kThreads && (1 << cover->lanes_log2) < (chunks > least ? chunks : least)) ++cover->lanes_log2;
    // wide rows in pieces of 256 down to 32 threads, whichever leaves the fewest idle (513 chunks: 17 of 32, not 3 of 256, 8192 x 4097)
    if (chunks > 32) {
        int64_t least_work = INT64_MAX;
        for (int log2 = 8; log2 >= 5; --log2) {
            const int64_t work = (chunks + (1ll << log2) - 1) >> log2 << log2;
            if (work < least_work) least_work = work, cover->lanes_log2 = log2;
        }
    }
    const int lanes = 1 << cover->lanes_log2;
    const int64_t across = (chunks + lanes - 1) / lanes, per_block = kThreads / lanes, down = (m + per_block - 1) / per_block;
    int64_t rows = (static_cast<int64_t>(num_sms) * resident + across - 1) / across;
    if (rows > down) rows = down;
    if (rows > 65535) rows = 65535;
    return dim3(static_cast<unsigned>(across), static_cast<unsigned>(rows), 1);
}

bool whole_chunks(const void *p, int64_t ld, int64_t m, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (m == 1 || ld * static_cast<int64_t>(size) % 16 == 0);
}

template <int kT, bool kGrad, int kQM>
cudaError_t launch_from(const void *dy, int64_t lddy, const Kept &p, int act, void *out, int64_t ldo, int num_sms, cudaStream_t stream) {
    const Activation a = activation_of(act);
    constexpr size_t kE = kT == ELEM_F32 ? 4 : 2;
    Cover cover;
    if (p.h % kChunk == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && whole_chunks(out, ldo, p.m, kE) && (!kGrad || whole_chunks(dy, lddy, p.m, kE))) {
        const dim3 grid = cover_rows(p.h / kChunk, 1, p.m, num_sms, kGrad ? kGradBlocks : kFromBlocks, &cover);
        return launch(from_kept_kernel<kT, kGrad, kQM>, grid, kThreads, stream, dy, lddy, p, a, out, ldo, cover);
    }
    // (a row may begin inside its first chunk)
    const dim3 grid = cover_rows((p.h + 2 * kChunk - 2) / kChunk, 1, p.m, num_sms, 16, &cover);
    return launch(from_kept_any_kernel<kT, kGrad, kQM>, grid, kThreads, stream, dy, lddy, p, a, out, ldo, cover);
}

template <int kT, bool kGrad>
cudaError_t launch_from(const void *dy, int64_t lddy, const Kept &p, int act, void *out, int64_t ldo, int num_sms, cudaStream_t stream) {
    switch (p.qmode) {
        case QM_TOKEN: return launch_from<kT, kGrad, QM_TOKEN>(dy, lddy, p, act, out, ldo, num_sms, stream);
        case QM_GROUP: return launch_from<kT, kGrad, QM_GROUP>(dy, lddy, p, act, out, ldo, num_sms, stream);
        default: return launch_from<kT, kGrad, QM_MX>(dy, lddy, p, act, out, ldo, num_sms, stream);
    }
}

template <int kT>
cudaError_t launch_to(const void *z, int64_t ldz, const Kept &p, int act, int num_sms, cudaStream_t stream) {
    const Activation a = activation_of(act);
    constexpr size_t kE = kT == ELEM_F32 ? 4 : 2;
    const int chunks = p.h / kChunk;
    if (p.h % kChunk == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && whole_chunks(z, ldz, p.m, kE) &&
        (p.qmode != QM_TOKEN || chunks <= 4 * 1024)) {
        Cover cover;
        if (p.qmode == QM_GROUP)
            return launch(act_quant_kernel<kT, QM_GROUP>, cover_rows(chunks, 16, p.m, num_sms, kToBlocks, &cover), kThreads, stream, z, ldz, p, a, cover);
        if (p.qmode == QM_MX)
            return launch(act_quant_kernel<kT, QM_MX>, cover_rows(chunks, 4, p.m, num_sms, kToBlocks, &cover), kThreads, stream, z, ldz, p, a, cover);
        if (chunks <= 32)
            return launch(act_quant_kernel<kT, QM_TOKEN>, cover_rows(chunks, 1, p.m, num_sms, kToBlocks, &cover), kThreads, stream, z, ldz, p, a, cover);
        // few rows: more threads a row; many: more chunks a thread
        const int v = p.m > 2 * num_sms || chunks > 2048 ? 4 : (chunks > 1024 ? 2 : 1);
        const int threads = ((chunks + v - 1) / v + 31) / 32 * 32;
        const dim3 grid(static_cast<unsigned>(p.m), 1, 1), warps(static_cast<unsigned>((p.m + kWarps - 1) / kWarps), 1, 1);
        if (v == 4 && chunks <= 64) return launch(act_quant_row_kernel<kT, 2, true>, warps, kThreads, stream, z, ldz, p, a);
        if (v == 4 && chunks <= 128) return launch(act_quant_row_kernel<kT, 4, true>, warps, kThreads, stream, z, ldz, p, a);
        switch (v) {
            case 1: return launch(act_quant_row_kernel<kT, 1, false>, grid, threads, stream, z, ldz, p, a);
            case 2: return launch(act_quant_row_kernel<kT, 2, false>, grid, threads, stream, z, ldz, p, a);
            default: return launch(act_quant_row_kernel<kT, 4, false>, grid, threads, stream, z, ldz, p, a);
        }
    }
    const int64_t units = (p.m * ((p.h + 127) / 128) + kWarps - 1) / kWarps, most = 64ll * num_sms;
    const dim3 spread(static_cast<unsigned>(units < most ? units : most), 1, 1);
    if (p.qmode == QM_GROUP) return launch(act_quant_any_kernel<kT, QM_GROUP, false>, spread, kThreads, stream, z, ldz, p, a);
    if (p.qmode == QM_MX) return launch(act_quant_any_kernel<kT, QM_MX, false>, spread, kThreads, stream, z, ldz, p, a);
    if (p.h <= 1024 && p.m > num_sms)
        return launch(act_quant_any_kernel<kT, QM_TOKEN, false>, dim3(static_cast<unsigned>((p.m + kWarps - 1) / kWarps), 1, 1), kThreads, stream, z,
                      ldz, p, a);
    return launch(act_quant_any_kernel<kT, QM_TOKEN, true>, dim3(static_cast<unsigned>(p.m), 1, 1), kThreads, stream, z, ldz, p, a);
}

}  // namespace

cudaError_t launch_act_quant(int kind, const void *z, int64_t ldz, const Kept &to, int act, int num_sms, cudaStream_t stream) {
    switch (kind) {
        case ELEM_F16: return launch_to<ELEM_F16>(z, ldz, to, act, num_sms, stream);
        case ELEM_BF16: return launch_to<ELEM_BF16>(z, ldz, to, act, num_sms, stream);
        default: return launch_to<ELEM_F32>(z, ldz, to, act, num_sms, stream);
    }
}

cudaError_t launch_act_dequant(int kind, const Kept &from, int act, void *out, int64_t ldo, int num_sms, cudaStream_t stream) {
    switch (kind) {
        case ELEM_F16: return launch_from<ELEM_F16, false>(nullptr, 0, from, act, out, ldo, num_sms, stream);
        case ELEM_BF16: return launch_from<ELEM_BF16, false>(nullptr, 0, from, act, out, ldo, num_sms, stream);
        default: return launch_from<ELEM_F32, false>(nullptr, 0, from, act, out, ldo, num_sms, stream);
    }
}

cudaError_t launch_act_grad_quant(bool bf16, const void *dy, int64_t lddy, const Kept &z, int act, void *dz, int64_t lddz,
                                  int num_sms, cudaStream_t stream) {
    return bf16 ? launch_from<ELEM_BF16, true>(dy, lddy, z, act, dz, lddz, num_sms, stream)
                : launch_from<ELEM_F16, true>(dy, lddy, z, act, dz, lddz, num_sms, stream);
}

}  // namespace mc2
