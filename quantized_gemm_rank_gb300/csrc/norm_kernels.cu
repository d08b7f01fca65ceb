// norm_kernels.cu -- residual RMS norm with optional 8-bit output, and its
// gradient.
//
//   s[t, j]  = x[t, j] + residual[t, j]                (or x, without a residual)
//   rstd[t]  = 1 / sqrt(mean_j s[t, j]^2 + eps)
//   y[t, j]  = s[t, j] * rstd[t] * weight[j]
// out is y and residual_out is s, each rounded once; the 8-bit codes are made
// from the unrounded y.  Bound by memory: each row is read once and kept in
// registers between its sum, its largest value and its outputs (4096 x 8192 bf16
// with residual: 41.0 us, 6.5 TB/s, to 16 bits; 40.9 us, 5.7 TB/s, to int8).
//
//   xhat = s * rstd,  g = dy * weight,  c[t] = mean_j g[t, j] xhat[t, j]
//   dx[t, j] = rstd[t] (g[t, j] - xhat[t, j] c[t]) (+ dres[t, j])
//   dw[j]    = sum_t dy[t, j] xhat[t, j]
#include "norm.h"

#include "host.h"
#include "internal.h"
#include "num.cuh"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kNormGradStages = 6;

// Blocks of the gradient that share an SM: 1024 threads, a vector each, at most 8 blocks
// (8192 x 4096: 49.0 us, against 70.0 with 512 threads an SM and 66.6 with 2048, whose
// rings are too short; 32768 x 1024: 49.9, 67.3 and 49.9).
int norm_grad_blocks_per_sm(int64_t h, int elem_size) {
    const int64_t threads = (h * elem_size / 16 + 31) / 32 * 32;
    const int64_t blocks = 1024 / (threads > 0 ? threads : 32);
    return static_cast<int>(blocks < 1 ? 1 : (blocks > 8 ? 8 : blocks));
}

constexpr uint32_t kGradSmem = 216 * 1024;   // of an SM, for the gradient's rings
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sum over the block, the same value and the same order in every thread.
__device__ __forceinline__ float block_sum(float v, float *slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += slots[w];
    return s;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, float *slots) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = __uint_as_float(v);
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s = max(s, __float_as_uint(slots[w]));
    return s;
}

__device__ __forceinline__ float weight_at(const void *w, int w_f32, int j, int kT) {
    if (w_f32) return static_cast<const float *>(w)[j];
    if (kT == ELEM_F16) return Elem<ELEM_F16>::load(static_cast<const __half *>(w) + j);
    return Elem<ELEM_BF16>::load(static_cast<const __nv_bfloat16 *>(w) + j);
}

// ------------------------------------------------------------------ rows in registers
// Rows that are whole 16-byte vectors are read once and kept: thread t of T holds
// vectors t, t + T, ..., V of them, so neighbouring lanes hold neighbouring
// vectors and a group of 32 or 128 elements is 4 to 32 consecutive lanes.

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

// The weights of vector c, of x's type or fp32.
template <int kT>
__device__ __forceinline__ void load_weights(const void *w, int w_f32, int c, float (&f)[Vec<kT>::kW]) {
    if (kT == ELEM_F32 || !w_f32) {
        unpack<kT>(__ldg(static_cast<const uint4 *>(w) + c), f);
    } else {
#pragma unroll
        for (int i = 0; i < Vec<kT>::kW / 4; ++i) {
            const float4 v = __ldg(static_cast<const float4 *>(w) + c * (Vec<kT>::kW / 4) + i);
            f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
        }
    }
}

// The larger of a and |b|; a NaN is kept.
__device__ __forceinline__ float max_abs(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// Sum and largest value over the block: one barrier each, the warps' values in
// slots of their own, and the same tree in every warp (so every thread has the same bits).
__device__ __forceinline__ float block_sum32(float v, float *slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (blockDim.x == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (blockDim.x >> 5) ? slots[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

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

// One row a block, V vectors a thread.
template <int kT, int V, int kQM>
__global__ void __launch_bounds__(1024) norm_row_kernel(const __grid_constant__ NormParams p) {
    constexpr int kW = Vec<kT>::kW;
    constexpr int kE = kT == ELEM_F32 ? 4 : 2;
    __shared__ float sum_slots[32];
    __shared__ uint32_t max_slots[32];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int64_t row = blockIdx.x;
    const int T = blockDim.x, nv = p.h / kW;
    const char *x = static_cast<const char *>(p.x) + row * p.ldx * kE;
    const char *res = p.res ? static_cast<const char *>(p.res) + row * p.ldr * kE : nullptr;
    uint4 raw[V], add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        raw[i] = add[i] = make_uint4(0, 0, 0, 0);
        if (c < nv) {
            raw[i] = load_once(x + static_cast<int64_t>(c) * 16);
            if (res) add[i] = load_once(res + static_cast<int64_t>(c) * 16);
        }
    }
    float s[V][kW];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float r[kW];
        unpack<kT>(raw[i], s[i]);
        unpack<kT>(add[i], r);
#pragma unroll
        for (int e = 0; e < kW; ++e) {
            if (res) s[i][e] = __fadd_rn(s[i][e], r[e]);
            ss = fmaf(s[i][e], s[i][e], ss);
        }
        const int c = threadIdx.x + i * T;
        if (p.res_out && c < nv)
            *reinterpret_cast<uint4 *>(static_cast<char *>(p.res_out) + row * p.ldro * kE + static_cast<int64_t>(c) * 16) =
                pack<kT>(s[i]);
    }
    const float rstd = rsqrtf(block_sum32(ss, sum_slots) / static_cast<float>(p.h) + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        float w[kW];
        if (c < nv) {
            load_weights<kT>(p.w, p.w_f32, c, w);
        } else {
#pragma unroll
            for (int e = 0; e < kW; ++e) w[e] = 0.0f;
        }
        float largest = 0.0f;
#pragma unroll
        for (int e = 0; e < kW; ++e) {
            s[i][e] = s[i][e] * rstd * w[e];
            if (c >= nv) s[i][e] = 0.0f;   // (an infinite rstd times zero)
            if constexpr (kQM != QM_NONE) largest = max_abs(largest, s[i][e]);
        }
        uint32_t a = __float_as_uint(largest);   // of non-negative values: ordered like them
        if (p.out && c < nv)
            *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + row * p.ldo * kE + static_cast<int64_t>(c) * 16) =
                pack<kT>(s[i]);
        if constexpr (kQM == QM_TOKEN) top = max(top, a);
        if constexpr (kQM == QM_GROUP || kQM == QM_MX) {
            constexpr int kG = kQM == QM_GROUP ? 128 : 32;
#pragma unroll
            for (int o = kG / kW / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
            const bool first = (threadIdx.x & (kG / kW - 1)) == 0 && c < nv;
            const int64_t at = row * ((p.h + kG - 1) / kG) + c / (kG / kW);
            float r[kW];
            if constexpr (kQM == QM_GROUP) {
                const float step = __fdiv_rn(__uint_as_float(a), q_max(p.qkind));
                if (first) static_cast<float *>(p.scale)[at] = step;
                quotients(s[i], step, r);
            } else {
                const uint32_t code = mx_code(a, p.qkind);
                if (first) static_cast<uint8_t *>(p.scale)[at] = static_cast<uint8_t>(code);
                const float inverse = mx_inverse(code);
#pragma unroll
                for (int e = 0; e < kW; ++e) r[e] = code != 0xFFu ? s[i][e] * inverse : 0.0f;
            }
            if (c < nv) store_codes(p.q, row * p.h + static_cast<int64_t>(c) * kW, r, p.qkind);
        }
    }
    if constexpr (kQM == QM_TOKEN) {
        const float step = __fdiv_rn(__uint_as_float(block_max32(top, max_slots)), q_max(p.qkind));
        if (threadIdx.x == 0) static_cast<float *>(p.scale)[row] = step;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            float r[kW];
            quotients(s[i], step, r);
            if (c < nv) store_codes(p.q, row * p.h + static_cast<int64_t>(c) * kW, r, p.qkind);
        }
    }
}

// Gradient, V vectors a thread.  Block b takes rows b, b + B, ... and keeps its share
// of dw in registers.  A row's sum c stands between its reads and its
// writes, so the rows come through a ring of bulk copies in shared memory: those
// behind the one at work are on their way while it waits for its barrier (read
// straight to registers one row ahead: 98.4 us for 8192 x 8192 bf16, dw included, against 90.3: 5.9 TB/s).
template <int kT, int V>
__global__ void __launch_bounds__(1024) norm_grad_row_kernel(const __grid_constant__ NormGradParams p, int stages,
                                                            int *status, uint64_t wait_limit_ns) {
    constexpr int kW = Vec<kT>::kW;
    constexpr int kE = kT == ELEM_F32 ? 4 : 2;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float slots[2][32];
    __shared__ __align__(8) uint64_t full[kNormGradStages];
    const int T = blockDim.x, nv = p.h / kW;
    const uint32_t row_bytes = static_cast<uint32_t>(p.h) * kE;
    const uint32_t stage_bytes = row_bytes * (p.dres ? 3 : 2);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) ptx::mbar_init(ptx::smem_u32(&full[i]), 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    auto fetch = [&](int64_t row, int stage) {   // one thread
        const uint32_t bar = ptx::smem_u32(&full[stage]);
        const uint32_t to = ptx::smem_u32(ring) + stage * stage_bytes;
        ptx::mbar_arrive_expect_tx(bar, stage_bytes);
        ptx::bulk_load_1d(to, static_cast<const char *>(p.x) + row * p.ldx * kE, row_bytes, bar);
        ptx::bulk_load_1d(to + row_bytes, static_cast<const char *>(p.dy) + row * p.lddy * kE, row_bytes, bar);
        if (p.dres)
            ptx::bulk_load_1d(to + 2 * row_bytes, static_cast<const char *>(p.dres) + row * p.lddres * kE, row_bytes, bar);
    };
    const int64_t first = blockIdx.x, step = gridDim.x;
    if (threadIdx.x == 0)
        for (int i = 0; i < stages && first + i * step < p.m; ++i) fetch(first + i * step, i);
    float dw[V][kW];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < kW; ++e) dw[i][e] = 0.0f;
    // the weights stay in registers in 16 bits (beside the ring L1 has no room for them);
    // with two vectors a thread, or in fp32 beside 16-bit rows, they are read again for each row
    constexpr bool kKeep = V == 1;
    const bool kept = kKeep && (kT == ELEM_F32 || !p.w_f32);
    uint4 wr = make_uint4(0, 0, 0, 0);
    if (kept && threadIdx.x < nv) wr = __ldg(static_cast<const uint4 *>(p.w) + threadIdx.x);
    auto weights = [&](int k, float (&w)[kW]) {
        if (kept)
            unpack<kT>(wr, w);
        else
            load_weights<kT>(p.w, p.w_f32, k, w);
    };
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    float next_rstd = p.rstd[first];
    bool failed = false;
    for (int64_t row = first; row < p.m; row += step, turn ^= 1) {
        const float rstd = next_rstd;
        if (row + step < p.m) next_rstd = p.rstd[row + step];
        failed = !ptx::mbar_wait(ptx::smem_u32(&full[stage]), phase, wait_limit_ns);
        const uint4 *xs = reinterpret_cast<const uint4 *>(ring + stage * stage_bytes);
        const uint4 *ds = reinterpret_cast<const uint4 *>(ring + stage * stage_bytes + row_bytes);
        const uint4 *as = reinterpret_cast<const uint4 *>(ring + stage * stage_bytes + 2 * row_bytes);
        float c = 0.0f;
        // with one vector a thread its values stay in registers over the barrier
        float xhat[kW], gw[kW];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = threadIdx.x + i * T;
            if (k < nv && !failed) {
                float w[kW];
                unpack<kT>(xs[k], xhat);
                unpack<kT>(ds[k], gw);
                weights(k, w);
#pragma unroll
                for (int e = 0; e < kW; ++e) {
                    xhat[e] *= rstd;
                    dw[i][e] = fmaf(gw[e], xhat[e], dw[i][e]);
                    gw[e] *= w[e];
                    c = fmaf(gw[e], xhat[e], c);
                }
            }
        }
        // the row's sum; the slots alternate, so a warp that is a row ahead does not
        // overwrite what another still reads
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        bool any;
        if (T > 32) {
            const int lane = threadIdx.x & 31;
            if (lane == 0) slots[turn][threadIdx.x >> 5] = c;
            any = __syncthreads_or(failed);
            c = lane < (T >> 5) ? slots[turn][lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        } else {
            any = __any_sync(0xFFFFFFFFu, failed);
            __syncwarp();   // (a vote orders no memory: the lanes' reads of the row before, ahead of the copy that replaces it)
        }
        if (any) {
            // a copy did not arrive in time: the launch is given up, once those in flight have had time to land
            if (threadIdx.x == 0 && status) atomicExch(status, -7);
            ptx::nanosleep(20000);
            return;
        }
        c /= static_cast<float>(p.h);
        // every thread is past the row before this one: its stage takes the next row
        if (threadIdx.x == 0 && row != first) {
            const int64_t next = row + (stages - 1) * step;
            if (next < p.m) fetch(next, stage == 0 ? stages - 1 : stage - 1);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = threadIdx.x + i * T;
            if (k < nv) {
                float a[kW];
                if constexpr (!kKeep) {
                    float w[kW];
                    unpack<kT>(xs[k], xhat);
                    unpack<kT>(ds[k], gw);
                    weights(k, w);
#pragma unroll
                    for (int e = 0; e < kW; ++e) {
                        xhat[e] *= rstd;
                        gw[e] *= w[e];
                    }
                }
                if (p.dres) unpack<kT>(as[k], a);
#pragma unroll
                for (int e = 0; e < kW; ++e) {
                    const float d = gw[e] - xhat[e] * c;
                    a[e] = p.dres ? fmaf(rstd, d, a[e]) : rstd * d;
                }
                *reinterpret_cast<uint4 *>(static_cast<char *>(p.dx) + row * p.lddx * kE + static_cast<int64_t>(k) * 16) =
                    pack<kT>(a);
            }
        }
        if (++stage == stages) stage = 0, phase ^= 1u;
    }
    if (p.dw) {
        float *part = p.parts + static_cast<int64_t>(blockIdx.x) * p.h;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = threadIdx.x + i * T;
            if (k < nv)
#pragma unroll
                for (int e = 0; e < kW; e += 4)
                    *reinterpret_cast<float4 *>(part + k * kW + e) =
                        make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
        }
    }
}

// ------------------------------------------------------------------ any layout
// Rows that are not whole 16-byte vectors: the row in registers too, by element loads.  A
// warp takes blocks of 128 elements, V of them, lane l elements l, l + 32, l + 64 and
// l + 96, so a group's largest value is found in one warp.
template <int kT, int V>
__global__ void __launch_bounds__(1024, 1) norm_odd_kernel(const __grid_constant__ NormParams p) {
    using T = typename Elem<kT>::type;
    __shared__ float sum_slots[32];
    __shared__ uint32_t max_slots[32];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.res ? static_cast<const T *>(p.res) + row * p.ldr : nullptr;
    auto at = [&](int i, int e) { return (warp + i * warps) * 128 + 32 * e + lane; };
    float s[V][4], w[V][4];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = at(i, e);
            s[i][e] = w[i][e] = 0.0f;
            if (j < p.h) {
                s[i][e] = Elem<kT>::load(x + j);
                if (res) s[i][e] = __fadd_rn(s[i][e], Elem<kT>::load(res + j));
                w[i][e] = weight_at(p.w, p.w_f32, j, kT);
            }
        }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(s[i][e], s[i][e], ss);
    const float rstd = rsqrtf(block_sum32(ss, sum_slots) / static_cast<float>(p.h) + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    T *out = p.out ? static_cast<T *>(p.out) + row * p.ldo : nullptr;
    T *ro = p.res_out ? static_cast<T *>(p.res_out) + row * p.ldro : nullptr;
    float largest = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = at(i, e);
            if (j < p.h) {
                if (ro) Elem<kT>::store(ro + j, s[i][e]);
                s[i][e] = s[i][e] * rstd * w[i][e];
                if (out) Elem<kT>::store(out + j, s[i][e]);
                largest = max_abs(largest, s[i][e]);
            } else {
                s[i][e] = 0.0f;   // (an infinite rstd times zero)
            }
        }
    if (p.qmode == QM_NONE) return;
    float token = 0.0f;
    if (p.qmode == QM_TOKEN) {
        token = __fdiv_rn(__uint_as_float(block_max32(__float_as_uint(largest), max_slots)), q_max(p.qkind));
        if (threadIdx.x == 0) static_cast<float *>(p.scale)[row] = token;
    }
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.h;
    const int groups = p.qmode == QM_MX ? (p.h + 31) / 32 : (p.h + 127) / 128;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int block = warp + i * warps;
        if (block * 128 >= p.h) break;   // (the same in the whole warp)
        float r[4];
        if (p.qmode == QM_MX) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t code = mx_code(__reduce_max_sync(0xFFFFFFFFu, abs_bits(s[i][e])), p.qkind);
                if (lane == 0 && block * 4 + e < groups)
                    static_cast<uint8_t *>(p.scale)[row * groups + block * 4 + e] = static_cast<uint8_t>(code);
                r[e] = code != 0xFFu ? s[i][e] * mx_inverse(code) : 0.0f;
            }
        } else {
            float step = token;
            if (p.qmode == QM_GROUP) {
                uint32_t a = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) a = max(a, abs_bits(s[i][e]));
                step = __fdiv_rn(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, a)), q_max(p.qkind));
                if (lane == 0) static_cast<float *>(p.scale)[row * groups + block] = step;
            }
            quotients(s[i], step, r);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = at(i, e);
            if (j < p.h) q[j] = static_cast<uint8_t>(encode8(r[e], p.qkind));
        }
    }
}

// Gradient of such rows: block b takes rows b, b + B, ..., its share of dw in registers, E
// columns a thread; x and dy are read twice (the second time from L1).
template <int kT, int E>
__global__ void __launch_bounds__(1024, 1) norm_grad_odd_kernel(const __grid_constant__ NormGradParams p) {
    using T = typename Elem<kT>::type;
    __shared__ float slots[2][32];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    float dw[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = 0.0f;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x, turn ^= 1) {
        const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *dres = p.dres ? static_cast<const T *>(p.dres) + row * p.lddres : nullptr;
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
        const float rstd = p.rstd[row];
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i % 4 == 0) asm volatile("" ::: "memory");   // (four columns' loads at once: more do not fit the registers)
            const int j = threadIdx.x + i * blockDim.x;
            if (j < p.h) {
                const float xhat = Elem<kT>::load(x + j) * rstd, d = Elem<kT>::load(dy + j);
                dw[i] = fmaf(d, xhat, dw[i]);
                c = fmaf(d * weight_at(p.w, p.w_f32, j, kT), xhat, c);
            }
        }
        c = block_sum32(c, slots[turn]) / static_cast<float>(p.h);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i % 4 == 0) asm volatile("" ::: "memory");
            const int j = threadIdx.x + i * blockDim.x;
            if (j < p.h) {
                const float xhat = Elem<kT>::load(x + j) * rstd;
                const float g = Elem<kT>::load(dy + j) * weight_at(p.w, p.w_f32, j, kT);
                const float d = g - xhat * c;
                Elem<kT>::store(dx + j, dres ? fmaf(rstd, d, Elem<kT>::load(dres + j)) : rstd * d);
            }
        }
    }
    if (p.dw) {
        float *part = p.parts + static_cast<int64_t>(blockIdx.x) * p.h;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < p.h) part[j] = dw[i];
        }
    }
}

// Any sizes, strides and alignments: one block a row, the row re-read for each
// pass (statistics, largest value, outputs).  A warp takes whole groups of 32 or
// 128 elements, so that a group's scale is found inside one warp; the thread
// that reads an element in the last pass is the one that writes it, so outputs
// may overwrite x or residual.
template <int kT>
__global__ void __launch_bounds__(kThreads) norm_any_kernel(const __grid_constant__ NormParams p) {
    using T = typename Elem<kT>::type;
    __shared__ float slots[kWarps];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.res ? static_cast<const T *>(p.res) + row * p.ldr : nullptr;
    const int group = p.qmode == QM_MX ? 32 : 128;
    const int per_lane = group / 32;
    auto s_at = [&](int j) {
        float v = Elem<kT>::load(x + j);
        if (res) v = __fadd_rn(v, Elem<kT>::load(res + j));
        return v;
    };
    auto each = [&](auto f) {
        for (int g = warp * group; g < p.h; g += kWarps * group)
            for (int i = 0; i < per_lane; ++i) {
                const int j = g + 32 * i + lane;
                if (j < p.h) f(j);
            }
    };
    float ss = 0.0f;
    each([&](int j) {
        const float v = s_at(j);
        ss = fmaf(v, v, ss);
    });
    const float rstd = rsqrtf(block_sum(ss, slots) / static_cast<float>(p.h) + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    auto y_of = [&](float v, int j) { return v * rstd * weight_at(p.w, p.w_f32, j, kT); };
    float scale = 0.0f;
    if (p.qmode == QM_TOKEN) {
        uint32_t a = 0;
        each([&](int j) { a = max(a, abs_bits(y_of(s_at(j), j))); });
        scale = __fdiv_rn(__uint_as_float(block_max(a, slots)), q_max(p.qkind));
        if (threadIdx.x == 0) static_cast<float *>(p.scale)[row] = scale;
    }
    T *out = p.out ? static_cast<T *>(p.out) + row * p.ldo : nullptr;
    T *ro = p.res_out ? static_cast<T *>(p.res_out) + row * p.ldro : nullptr;
    uint8_t *q = p.q ? static_cast<uint8_t *>(p.q) + row * p.h : nullptr;
    const int groups = (p.h + group - 1) / group;
    for (int g = warp; g < groups; g += kWarps) {
        float y[4];
        uint32_t a = 0;
        for (int i = 0; i < per_lane; ++i) {
            const int j = g * group + 32 * i + lane;
            y[i] = 0.0f;
            if (j < p.h) {
                const float v = s_at(j);
                y[i] = y_of(v, j);
                if (ro) Elem<kT>::store(ro + j, v);
                if (out) Elem<kT>::store(out + j, y[i]);
                a = max(a, abs_bits(y[i]));
            }
        }
        if (p.qmode == QM_NONE) continue;
        a = __reduce_max_sync(0xFFFFFFFFu, a);
        float inverse = 0.0f, step = scale;
        bool live;
        if (p.qmode == QM_MX) {
            const uint32_t code = mx_code(a, p.qkind);
            if (lane == 0) static_cast<uint8_t *>(p.scale)[row * groups + g] = static_cast<uint8_t>(code);
            live = code != 0xFFu;
            inverse = mx_inverse(code);
        } else {
            if (p.qmode == QM_GROUP) {
                step = __fdiv_rn(__uint_as_float(a), q_max(p.qkind));
                if (lane == 0) static_cast<float *>(p.scale)[row * groups + g] = step;
            }
            live = usable(step);
        }
        for (int i = 0; i < per_lane; ++i) {
            const int j = g * group + 32 * i + lane;
            if (j < p.h)
                q[j] = live ? static_cast<uint8_t>(
                                  encode8(p.qmode == QM_MX ? y[i] * inverse : __fdiv_rn(y[i], step), p.qkind))
                            : 0;
        }
    }
}

// Gradient, any sizes, strides and alignments: block b takes rows b, b + B, ...
// and keeps its share of dw in its row of the workspace (each column is one
// thread's, so nothing races); dw_sum_kernel adds the B shares in order.
template <int kT>
__global__ void __launch_bounds__(kThreads) norm_grad_any_kernel(const __grid_constant__ NormGradParams p) {
    using T = typename Elem<kT>::type;
    __shared__ float slots[kWarps];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    float *part = p.dw ? p.parts + static_cast<int64_t>(blockIdx.x) * p.h : nullptr;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *dres = p.dres ? static_cast<const T *>(p.dres) + row * p.lddres : nullptr;
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
        const float rstd = p.rstd[row];
        float c = 0.0f;
        for (int j = threadIdx.x; j < p.h; j += kThreads) {
            const float xhat = Elem<kT>::load(x + j) * rstd;
            const float d = Elem<kT>::load(dy + j);
            c = fmaf(d * weight_at(p.w, p.w_f32, j, kT), xhat, c);
            if (part) part[j] = first ? d * xhat : fmaf(d, xhat, part[j]);
        }
        c = block_sum(c, slots) / static_cast<float>(p.h);
        for (int j = threadIdx.x; j < p.h; j += kThreads) {
            const float xhat = Elem<kT>::load(x + j) * rstd;
            const float g = Elem<kT>::load(dy + j) * weight_at(p.w, p.w_f32, j, kT);
            float v = rstd * (g - xhat * c);
            if (dres) v += Elem<kT>::load(dres + j);
            Elem<kT>::store(dx + j, v);
        }
        first = false;
    }
}

// dw from the blocks' shares: a block takes kCols columns, its 1024 / kCols groups of
// threads every so many-th share, added in order, and one warp a column the groups' sums, in
// a fixed tree.
template <int kCols>
__global__ void __launch_bounds__(1024) dw_sum_kernel(const float *parts, int count, int h, int w_kind, void *dw) {
    constexpr int kGroups = 1024 / kCols;
    __shared__ float sums[kGroups][kCols + 1];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int group = threadIdx.x / kCols, c = threadIdx.x % kCols;
    const int j0 = blockIdx.x * kCols;
    float s = 0.0f;
    if (j0 + c < h) {
#pragma unroll 10
        for (int b = group; b < count; b += kGroups) s += parts[static_cast<int64_t>(b) * h + j0 + c];
    }
    sums[group][c] = s;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = j0 + warp;
    if (warp >= kCols || j >= h) return;
    s = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; g += 32) s += sums[g + lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane != 0) return;
    if (w_kind == ELEM_F32)
        static_cast<float *>(dw)[j] = s;
    else if (w_kind == ELEM_F16)
        Elem<ELEM_F16>::store(static_cast<__half *>(dw) + j, s);
    else
        Elem<ELEM_BF16>::store(static_cast<__nv_bfloat16 *>(dw) + j, s);
}

template <class K, class... A>
cudaError_t launch(K kern, unsigned grid, unsigned block, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Whether rows can be read as whole 16-byte vectors.
bool vectors(const void *p, int64_t ld, int64_t m, int es) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (m == 1 || ld * es % 16 == 0));
}

template <int kT, int V>
cudaError_t norm_rows(const NormParams &p, unsigned threads, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.m);
    switch (p.qmode) {
        case QM_TOKEN: return launch(norm_row_kernel<kT, V, QM_TOKEN>, grid, threads, 0, stream, p);
        case QM_GROUP: return launch(norm_row_kernel<kT, V, QM_GROUP>, grid, threads, 0, stream, p);
        case QM_MX: return launch(norm_row_kernel<kT, V, QM_MX>, grid, threads, 0, stream, p);
        default: return launch(norm_row_kernel<kT, V, QM_NONE>, grid, threads, 0, stream, p);
    }
}

// Threads of a row of nv vectors at v a thread: whole warps, evenly filled.
unsigned row_threads(int nv, int v) { return static_cast<unsigned>((nv + 32 * v - 1) / (32 * v)) * 32; }

template <int kT>
cudaError_t norm(const NormParams &p, int num_sms, cudaStream_t stream) {
    constexpr int kW = Vec<kT>::kW, kE = 16 / kW;
    const int nv = p.h / kW;
    if (p.h % kW == 0 && nv <= 4 * 1024 && vectors(p.x, p.ldx, p.m, kE) && vectors(p.res, p.ldr, p.m, kE) &&
        vectors(p.out, p.ldo, p.m, kE) && vectors(p.res_out, p.ldro, p.m, kE) &&
        reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0) {
        // Rows that are all resident at once with one vector a thread are soonest done that way
        // (64 x 4096 to int8: 2.4 us, against 2.6 and 3.4 with 2 and 4).  More rows want more
        // blocks an SM, so that one's barriers are another's loads: 2 vectors without
        // codes (4096 x 8192: 46.4, 41.0 and 41.4 us with 1, 2 and 4), 4 with them, whose
        // second barrier and arithmetic lie between a row's loads and its stores (to
        // int8: 55.9, 50.0 and 40.9).
        const unsigned t1 = row_threads(nv, 1);
        int v = 4;
        if (nv <= 1024 && p.m <= static_cast<int64_t>(num_sms) * (2048 / t1))
            v = 1;
        else if (nv <= 2048 && p.qmode == QM_NONE)
            v = 2;
        if (v == 1) return norm_rows<kT, 1>(p, t1, stream);
        if (v == 2)   // (without codes)
            return launch(norm_row_kernel<kT, 2, QM_NONE>, static_cast<unsigned>(p.m), row_threads(nv, 2), 0, stream, p);
        return norm_rows<kT, 4>(p, row_threads(nv, 4), stream);
    }
    const unsigned grid = static_cast<unsigned>(p.m);
    const int blocks = (p.h + 127) / 128;   // a warp's
    if (blocks <= 32 && p.m <= static_cast<int64_t>(num_sms) * (64 / blocks))
        return launch(norm_odd_kernel<kT, 1>, grid, 32u * blocks, 0, stream, p);
    if (blocks <= 4 * 32) return launch(norm_odd_kernel<kT, 4>, grid, 32u * ((blocks + 3) / 4), 0, stream, p);
    return launch(norm_any_kernel<kT>, grid, kThreads, 0, stream, p);
}

template <int kT, int V>
cudaError_t norm_grad_rows(const NormGradParams &p, cudaStream_t stream) {
    constexpr int kW = Vec<kT>::kW, kE = 16 / kW;
    auto kern = norm_grad_row_kernel<kT, V>;
    thread_local unsigned long long ready_ctx = 0;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ctx != ready_ctx) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
        if (e != cudaSuccess) return e;
        ready_ctx = ctx;
    }
    const unsigned threads = row_threads(p.h / kW, V);
    const int parts = norm_grad_parts(p.m, p.h, kE);
    const uint32_t stage = static_cast<uint32_t>(p.h) * kE * (p.dres ? 3 : 2);
    // the blocks that share an SM share its memory; a block needs no more stages than it has rows
    const uint32_t room = kGradSmem / static_cast<uint32_t>(norm_grad_blocks_per_sm(p.h, kE));
    int stages = static_cast<int>(room / stage);
    const int64_t rows = (p.m + parts - 1) / parts;
    if (stages > kNormGradStages) stages = kNormGradStages;
    if (stages > rows) stages = static_cast<int>(rows);
    if (stages < 2) stages = 2;
    return launch(kern, static_cast<unsigned>(parts), threads, stages * stage, stream, p, stages, device_status_word(),
                  host::kWaitLimitNs);
}

template <int kT>
cudaError_t norm_grad(const NormGradParams &p, cudaStream_t stream) {
    constexpr int kW = Vec<kT>::kW, kE = 16 / kW;
    const int nv = p.h / kW;
    if (p.h % kW == 0 && nv <= 2048 && vectors(p.x, p.ldx, p.m, kE) && vectors(p.dy, p.lddy, p.m, kE) &&
        vectors(p.dres, p.lddres, p.m, kE) && vectors(p.dx, p.lddx, p.m, kE) &&
        reinterpret_cast<uintptr_t>(p.w) % 16 == 0)
        return nv <= 1024 ? norm_grad_rows<kT, 1>(p, stream) : norm_grad_rows<kT, 2>(p, stream);
    const unsigned grid = static_cast<unsigned>(norm_grad_parts(p.m, p.h, kE));
    if (p.h <= 4 * 1024) return launch(norm_grad_odd_kernel<kT, 4>, grid, row_threads(p.h, 4), 0, stream, p);
    if (p.h <= 8 * 1024) return launch(norm_grad_odd_kernel<kT, 8>, grid, row_threads(p.h, 8), 0, stream, p);
    if (p.h <= 16 * 1024) return launch(norm_grad_odd_kernel<kT, 16>, grid, row_threads(p.h, 16), 0, stream, p);
    return launch(norm_grad_any_kernel<kT>, grid, kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_add_rms_norm(int kind, const NormParams &p, int num_sms, cudaStream_t stream) {
    switch (kind) {
        case ELEM_F16: return norm<ELEM_F16>(p, num_sms, stream);
        case ELEM_BF16: return norm<ELEM_BF16>(p, num_sms, stream);
        default: return norm<ELEM_F32>(p, num_sms, stream);
    }
}

// (GB300's 152 SMs written out: the workspace's size is asked without a device.)
int norm_grad_parts(int64_t m, int64_t h, int elem_size) {
    const int64_t most = 152ll * norm_grad_blocks_per_sm(h, elem_size);
    return static_cast<int>(m < most ? m : most);
}

cudaError_t launch_rms_norm_grad(int kind, const NormGradParams &p, cudaStream_t stream) {
    switch (kind) {
        case ELEM_F16: return norm_grad<ELEM_F16>(p, stream);
        case ELEM_BF16: return norm_grad<ELEM_BF16>(p, stream);
        default: return norm_grad<ELEM_F32>(p, stream);
    }
}

cudaError_t launch_rms_norm_dw(int kind, const NormGradParams &p, cudaStream_t stream) {
    const float *parts = p.parts;
    const int count = norm_grad_parts(p.m, p.h, kind == ELEM_F32 ? 4 : 2), w_kind = p.w_f32 ? int(ELEM_F32) : kind;
    // narrow rows have many shares and few columns: 8 a block shortens each thread's sum
    // (300 x 512: 5.5 -> 4.4 us in all; 333 x 1000 4.4 -> 5.0, one row of 288 2.7 -> 3.3)
    if (p.h <= 512 && count > 64) return launch(dw_sum_kernel<8>, static_cast<unsigned>((p.h + 7) / 8), 1024, 0, stream, parts, count, p.h, w_kind, p.dw);
    return launch(dw_sum_kernel<32>, static_cast<unsigned>((p.h + 31) / 32), 1024, 0, stream, parts, count, p.h, w_kind, p.dw);
}

}  // namespace mc2
