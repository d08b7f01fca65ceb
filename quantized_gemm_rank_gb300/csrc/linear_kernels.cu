// linear_kernels.cu -- matrix product with bias, activation and residual in its
// epilogue, and the activation's derivative in the backward product.
//
//   z[i, j]   = sum_l x[i, l] W[l, j] + bias[j]
//   out[i, j] = act(z[i, j]) + residual[i, j],  preact = z        (forward)
//   out[i, j] = (sum_l x[i, l] W[l, j]) act'(aux[i, j])           (backward)
// Sums and the epilogue are fp32; each output is rounded once.
#include "linear.h"

#include "epilogue.cuh"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

// Any sizes, strides and alignments: a 64 x 64 tile a block, 4 x 4 outputs a
// thread, the operands staged through shared memory 16 columns at a time with
// element loads.
template <int kT>
__global__ void __launch_bounds__(256) linear_any_kernel(const __grid_constant__ LinearParams p, Activation act) {
    using T = typename Elem<kT>::type;
    __shared__ float xs[16][64 + 4], ws[16][64 + 4];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t n_tiles = (p.n + 63ll) / 64;
    const int m0 = static_cast<int>(blockIdx.x / n_tiles) * 64, n0 = static_cast<int>(blockIdx.x % n_tiles) * 64;
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + 256 * i, r = e >> 4, c = e & 15;
            xs[c][r] = (m0 + r < p.m && k0 + c < p.k) ? Elem<kT>::load(x + (m0 + r) * p.ldx + k0 + c) : 0.0f;
            if (p.w_nk) {
                ws[c][r] = (n0 + r < p.n && k0 + c < p.k) ? Elem<kT>::load(w + (n0 + r) * p.ldw + k0 + c) : 0.0f;
            } else {
                const int kr = e >> 6, nc = e & 63;
                ws[kr][nc] = (n0 + nc < p.n && k0 + kr < p.k) ? Elem<kT>::load(w + (k0 + kr) * p.ldw + n0 + nc) : 0.0f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int l = 0; l < 16; ++l) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = xs[l][ty * 4 + i], b[i] = ws[l][tx * 4 + i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
            if (r >= p.m || c >= p.n) continue;
            float z = acc[i][j];
            if (p.bias) z += Elem<kT>::load(static_cast<const T *>(p.bias) + c);
            if (p.preact) Elem<kT>::store(static_cast<T *>(p.preact) + r * p.ldp + c, z);
            const float aux = p.aux_mode != AUX_NONE ? Elem<kT>::load(static_cast<const T *>(p.aux) + r * p.ldaux + c) : 0.0f;
            const float o = p.aux_mode == AUX_ACT_GRAD ? z * act_derivative2(both(aux), act).x
                                                       : act2(both(z), act).x + (p.aux_mode == AUX_RESIDUAL ? aux : 0.0f);
            Elem<kT>::store(static_cast<T *>(p.out) + r * p.ldo + c, o);
        }
}

// Gradient through an activation alone, bound by memory: a thread takes eight columns (16
// bytes of each matrix) at a time where rows are whole vectors (8192 x 8192 with gelu: 64.3
// us, 6.3 TB/s), single elements otherwise.
template <bool kBF16>
__global__ void __launch_bounds__(256) act_grad_vec_kernel(const __grid_constant__ ActGradParams p, Activation act) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int64_t per_row = p.n / 8, total = p.m * per_row, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += step) {
        int64_t r = 0, c = e;
        if (p.m > 1) r = e / per_row, c = e - r * per_row;
        const uint4 d = *(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dy) + r * p.lddy) + c);
        const uint4 z = *(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.z) + r * p.ldz) + c);   // (may be dz: not the read-only path)
        float v[8];
        const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<kBF16>(dw[i]);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
        epilogue<kBF16, EPI_BACKWARD>(v, zw, act, true);
        *(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dz) + r * p.lddz) + c) =
            make_uint4(pack2<kBF16>(v[0], v[1]), pack2<kBF16>(v[2], v[3]), pack2<kBF16>(v[4], v[5]), pack2<kBF16>(v[6], v[7]));
    }
}

template <int kT>
__global__ void __launch_bounds__(256) act_grad_kernel(const __grid_constant__ ActGradParams p, Activation act) {
    using T = typename Elem<kT>::type;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int64_t total = p.m * p.n, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += step) {
        const int64_t r = e / p.n, c = e - r * p.n;
        const float d = Elem<kT>::load(static_cast<const T *>(p.dy) + r * p.lddy + c);
        const float z = Elem<kT>::load(static_cast<const T *>(p.z) + r * p.ldz + c);
        Elem<kT>::store(static_cast<T *>(p.dz) + r * p.lddz + c, d * act_derivative2(both(z), act).x);
    }
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

cudaError_t launch_linear_any(bool bf16, const LinearParams &p, cudaStream_t stream) {
    const int64_t tiles = ((p.m + 63ll) / 64) * ((p.n + 63ll) / 64);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    const Activation act = activation_of(p.act);
    return bf16 ? launch(linear_any_kernel<ELEM_BF16>, static_cast<unsigned>(tiles), 256, stream, p, act)
                : launch(linear_any_kernel<ELEM_F16>, static_cast<unsigned>(tiles), 256, stream, p, act);
}

cudaError_t launch_act_grad(bool bf16, const ActGradParams &in, int num_sms, cudaStream_t stream) {
    ActGradParams p = in;
    // matrices without gaps are one row
    if ((p.lddy == p.n && p.ldz == p.n && p.lddz == p.n) || p.m == 1) p.n *= p.m, p.m = 1;
    const Activation act = activation_of(p.act);
    const auto grid = [&](int64_t items) {
        const int64_t blocks = (items + 255) / 256, most = 64ll * num_sms;
        return static_cast<unsigned>(blocks < most ? blocks : most);
    };
    const auto vectors = [&](const void *q, int64_t ld) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && (p.m == 1 || ld % 8 == 0);
    };
    if (p.n % 8 == 0 && vectors(p.dy, p.lddy) && vectors(p.z, p.ldz) && vectors(p.dz, p.lddz))
        return bf16 ? launch(act_grad_vec_kernel<true>, grid(p.m * (p.n / 8)), 256, stream, p, act)
                    : launch(act_grad_vec_kernel<false>, grid(p.m * (p.n / 8)), 256, stream, p, act);
    return bf16 ? launch(act_grad_kernel<ELEM_BF16>, grid(p.m * p.n), 256, stream, p, act)
                : launch(act_grad_kernel<ELEM_F16>, grid(p.m * p.n), 256, stream, p, act);
}

}  // namespace mc2
