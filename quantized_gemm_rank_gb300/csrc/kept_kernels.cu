// kept_kernels.cu -- an activation kept in 8 bits, and what is made of it.
//
//   y = act(z),  scale = max|y| (1 / Q) over a row or a group,  q = y / scale to nearest-even    (act_quant)
//   out = act(q scale)                                                                           (act_dequant)
//   dz = dy act'(q scale)                                                                        (act_grad_quant)
// Arithmetic is fp32; codes and outputs are rounded once.
#include "kept.h"

#include "codes.cuh"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Any sizes, strides and alignments: one block a row, read once for its largest value and once for its codes.  A warp
// takes whole groups of 32 or 128 elements, so that a group's scale is found inside one warp.
template <int kT>
__global__ void __launch_bounds__(kThreads) act_quant_any_kernel(const void *z, int64_t ldz, const __grid_constant__ Kept p,
                                                                 Activation act) {
    using T = typename Elem<kT>::type;
    __shared__ uint32_t slots[32];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const T *from = static_cast<const T *>(z) + row * ldz;
    auto y_at = [&](int j) { return act2(both(Elem<kT>::load(from + j)), act).x; };
    float token = 0.0f;
    if (p.qmode == QM_TOKEN) {
        float top = 0.0f;
        for (int64_t j = threadIdx.x; j < p.h; j += kThreads) top = max_abs(top, y_at(static_cast<int>(j)));
        token = __fmul_rn(__uint_as_float(block_max32(__float_as_uint(top), slots)), q_inverse(p.qkind));
        if (threadIdx.x == 0) static_cast<float *>(p.scale)[row] = token;
    }
    const int group = p.qmode == QM_MX ? 32 : 128, groups = (p.h + group - 1) / group;
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.h;
    for (int g = warp; g < groups; g += kWarps) {
        float y[4];
        float top = 0.0f;
        for (int i = 0; i < group / 32; ++i) {
            const int j = g * group + 32 * i + lane;
            y[i] = j < p.h ? y_at(j) : 0.0f;
            top = max_abs(top, y[i]);
        }
        const uint32_t a = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
        float step = token, inverse = 0.0f;
        bool live;
        if (p.qmode == QM_MX) {
            const uint32_t code = mx_code(a, p.qkind);
            if (lane == 0) static_cast<uint8_t *>(p.scale)[row * groups + g] = static_cast<uint8_t>(code);
            live = code != 0xFFu;
            inverse = mx_inverse(code);
        } else {
            if (p.qmode == QM_GROUP) {
                step = __fmul_rn(__uint_as_float(a), q_inverse(p.qkind));
                if (lane == 0) static_cast<float *>(p.scale)[row * groups + g] = step;
            }
            live = usable(step);
        }
        for (int i = 0; i < group / 32; ++i) {
            const int j = g * group + 32 * i + lane;
            if (j < p.h)
                q[j] = live ? static_cast<uint8_t>(encode8(p.qmode == QM_MX ? y[i] * inverse : __fdiv_rn(y[i], step), p.qkind)) : 0;
        }
    }
}

// Element by element.
template <int kT, bool kGrad>
__global__ void __launch_bounds__(kThreads) from_kept_any_kernel(const void *dy, int64_t lddy, const __grid_constant__ Kept p,
                                                                 Activation act, void *out, int64_t ldo) {
    using T = typename Elem<kT>::type;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int64_t total = p.m * p.h, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < total; e += step) {
        const int64_t r = e / p.h;
        const int c = static_cast<int>(e - r * p.h);
        const float z = decode8(static_cast<const uint8_t *>(p.q)[e], p.qkind) * scale_at(p.scale, p.qmode, r, p.h, c);
        const float v = kGrad ? Elem<kT>::load(static_cast<const T *>(dy) + r * lddy + c) * act_derivative2(both(z), act).x
                              : act2(both(z), act).x;
        Elem<kT>::store(static_cast<T *>(out) + r * ldo + c, v);
    }
}

template <class K, class... A>
cudaError_t launch(K kern, unsigned grid, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned elementwise_grid(int64_t items, int num_sms) {
    const int64_t blocks = (items + kThreads - 1) / kThreads, most = 64ll * num_sms;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_act_quant(int kind, const void *z, int64_t ldz, const Kept &to, int act, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const Activation a = activation_of(act);
    const unsigned grid = static_cast<unsigned>(to.m);
    switch (kind) {
        case ELEM_F16: return launch(act_quant_any_kernel<ELEM_F16>, grid, stream, z, ldz, to, a);
        case ELEM_BF16: return launch(act_quant_any_kernel<ELEM_BF16>, grid, stream, z, ldz, to, a);
        default: return launch(act_quant_any_kernel<ELEM_F32>, grid, stream, z, ldz, to, a);
    }
}

cudaError_t launch_act_dequant(int kind, const Kept &from, int act, void *out, int64_t ldo, int num_sms, cudaStream_t stream) {
    const Activation a = activation_of(act);
    const unsigned grid = elementwise_grid(from.m * from.h, num_sms);
    const void *none = nullptr;
    const int64_t zero = 0;
    switch (kind) {
        case ELEM_F16: return launch(from_kept_any_kernel<ELEM_F16, false>, grid, stream, none, zero, from, a, out, ldo);
        case ELEM_BF16: return launch(from_kept_any_kernel<ELEM_BF16, false>, grid, stream, none, zero, from, a, out, ldo);
        default: return launch(from_kept_any_kernel<ELEM_F32, false>, grid, stream, none, zero, from, a, out, ldo);
    }
}

cudaError_t launch_act_grad_quant(bool bf16, const void *dy, int64_t lddy, const Kept &z, int act, void *dz, int64_t lddz,
                                  int num_sms, cudaStream_t stream) {
    const Activation a = activation_of(act);
    const unsigned grid = elementwise_grid(z.m * z.h, num_sms);
    return bf16 ? launch(from_kept_any_kernel<ELEM_BF16, true>, grid, stream, dy, lddy, z, a, dz, lddz)
                : launch(from_kept_any_kernel<ELEM_F16, true>, grid, stream, dy, lddy, z, a, dz, lddz);
}

}  // namespace mc2
