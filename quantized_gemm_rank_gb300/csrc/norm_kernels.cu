// norm_kernels.cu -- residual RMS norm with optional 8-bit output, and its
// gradient.
//
//   s[t, j]  = x[t, j] + residual[t, j]                (or x, without a residual)
//   rstd[t]  = 1 / sqrt(mean_j s[t, j]^2 + eps)
//   y[t, j]  = s[t, j] * rstd[t] * weight[j]
// out is y and residual_out is s, each rounded once; the 8-bit codes are made
// from the unrounded y.
//
//   xhat = s * rstd,  g = dy * weight,  c[t] = mean_j g[t, j] xhat[t, j]
//   dx[t, j] = rstd[t] (g[t, j] - xhat[t, j] c[t]) (+ dres[t, j])
//   dw[j]    = sum_t dy[t, j] xhat[t, j]
#include "norm.h"

#include "num.cuh"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

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

__device__ __forceinline__ float weight_at(const NormParams &p, int j, int kT) {
    if (p.w_f32) return static_cast<const float *>(p.w)[j];
    if (kT == ELEM_F16) return Elem<ELEM_F16>::load(static_cast<const __half *>(p.w) + j);
    return Elem<ELEM_BF16>::load(static_cast<const __nv_bfloat16 *>(p.w) + j);
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
    auto y_of = [&](float v, int j) { return v * rstd * weight_at(p, j, kT); };
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
            live = step > 0.0f;
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
    NormParams wp;
    wp.w = p.w;
    wp.w_f32 = p.w_f32;
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
            c = fmaf(d * weight_at(wp, j, kT), xhat, c);
            if (part) part[j] = first ? d * xhat : fmaf(d, xhat, part[j]);
        }
        c = block_sum(c, slots) / static_cast<float>(p.h);
        for (int j = threadIdx.x; j < p.h; j += kThreads) {
            const float xhat = Elem<kT>::load(x + j) * rstd;
            const float g = Elem<kT>::load(dy + j) * weight_at(wp, j, kT);
            float v = rstd * (g - xhat * c);
            if (dres) v += Elem<kT>::load(dres + j);
            Elem<kT>::store(dx + j, v);
        }
        first = false;
    }
}

__global__ void __launch_bounds__(kThreads) dw_sum_kernel(const float *parts, int count, int h, int w_kind, void *dw) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= h) return;
    float s = 0.0f;
    for (int b = 0; b < count; ++b) s += parts[static_cast<int64_t>(b) * h + j];
    if (w_kind == ELEM_F32)
        static_cast<float *>(dw)[j] = s;
    else if (w_kind == ELEM_F16)
        Elem<ELEM_F16>::store(static_cast<__half *>(dw) + j, s);
    else
        Elem<ELEM_BF16>::store(static_cast<__nv_bfloat16 *>(dw) + j, s);
}

template <class K, class... A>
cudaError_t launch(K kern, unsigned grid, unsigned block, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rms_norm(int kind, const NormParams &p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.m);
    switch (kind) {
        case ELEM_F16: return launch(norm_any_kernel<ELEM_F16>, grid, kThreads, stream, p);
        case ELEM_BF16: return launch(norm_any_kernel<ELEM_BF16>, grid, kThreads, stream, p);
        default: return launch(norm_any_kernel<ELEM_F32>, grid, kThreads, stream, p);
    }
}

int norm_grad_parts(int64_t m) { return static_cast<int>(m < kNormGradMaxParts ? m : kNormGradMaxParts); }

cudaError_t launch_rms_norm_grad(int kind, const NormGradParams &p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(norm_grad_parts(p.m));
    switch (kind) {
        case ELEM_F16: return launch(norm_grad_any_kernel<ELEM_F16>, grid, kThreads, stream, p);
        case ELEM_BF16: return launch(norm_grad_any_kernel<ELEM_BF16>, grid, kThreads, stream, p);
        default: return launch(norm_grad_any_kernel<ELEM_F32>, grid, kThreads, stream, p);
    }
}

cudaError_t launch_rms_norm_dw(int kind, const NormGradParams &p, cudaStream_t stream) {
    return launch(dw_sum_kernel, static_cast<unsigned>((p.h + kThreads - 1) / kThreads), kThreads, stream,
                  static_cast<const float *>(p.parts), norm_grad_parts(p.m), p.h, p.w_f32 ? int(ELEM_F32) : kind, p.dw);
}

}  // namespace mc2
