// quant_linear.cu -- products of 8-bit codes: the int8 product with scales per token and per channel, and the weight
// gradient whose input is kept in 8 bits.
//
//   out[t, j] = act(float(sum_l x[t, l] W[l, j]) x_scale[t] w_scale[j] + bias[j]) + residual[t, j]
//   dw[i, j]  = sum_t dy[t, i] act(q[t, j] scale),  db[i] = sum_t dy[t, i]
#include "kept.h"

#include "codes.cuh"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

// Any sizes, strides and alignments: a 64 x 64 tile a block, 4 x 4 outputs a thread, exact int32 sums.
template <int kT>
__global__ void __launch_bounds__(256) quant_product_any_kernel(const __grid_constant__ QuantProduct p, Activation act) {
    using T = typename Elem<kT>::type;
    __shared__ int xs[16][64 + 4], ws[16][64 + 4];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n_tiles = (p.n + 63) / 64;
    const int m0 = static_cast<int>(blockIdx.x / n_tiles) * 64, n0 = static_cast<int>(blockIdx.x % n_tiles) * 64;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.k; k0 += 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + 256 * i, r = e >> 4, c = e & 15;
            xs[c][r] = (m0 + r < p.m && k0 + c < p.k) ? p.x[(m0 + r) * p.ldx + k0 + c] : 0;
            if (p.w_nk) {
                ws[c][r] = (n0 + r < p.n && k0 + c < p.k) ? p.w[(n0 + r) * p.ldw + k0 + c] : 0;
            } else {
                const int kr = e >> 6, nc = e & 63;
                ws[kr][nc] = (n0 + nc < p.n && k0 + kr < p.k) ? p.w[(k0 + kr) * p.ldw + n0 + nc] : 0;
            }
        }
        __syncthreads();
#pragma unroll
        for (int l = 0; l < 16; ++l)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += xs[l][ty * 4 + i] * ws[l][tx * 4 + j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
            if (r >= p.m || c >= p.n) continue;
            float z = __fmul_rn(__fmul_rn(__int2float_rn(acc[i][j]), p.x_scale[r]), p.w_scale[c]);
            if (p.bias) z = __fadd_rn(z, p.bias_f32 ? static_cast<const float *>(p.bias)[c] : Elem<kT>::load(static_cast<const T *>(p.bias) + c));
            float o = act2(both(z), act).x;
            if (p.residual) o = __fadd_rn(o, Elem<kT>::load(static_cast<const T *>(p.residual) + r * p.ldr + c));
            Elem<kT>::store(static_cast<T *>(p.out) + r * p.ldo + c, o);
        }
}

// The same for the weight gradient; the blocks of the first column of tiles sum dy.
template <int kT>
__global__ void __launch_bounds__(256) quant_weight_grad_any_kernel(const __grid_constant__ QuantWeightGrad p, Activation act) {
    using T = typename Elem<kT>::type;
    __shared__ float ds[16][64 + 4], xs[16][64 + 4];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int k_tiles = (p.k + 63) / 64;
    const int i0 = static_cast<int>(blockIdx.x / k_tiles) * 64, j0 = static_cast<int>(blockIdx.x % k_tiles) * 64;
    float acc[4][4] = {}, sum = 0.0f;
    for (int t0 = 0; t0 < p.m; t0 += 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + 256 * i, t = e >> 6, c = e & 63;
            const int64_t row = t0 + t;
            ds[t][c] = (row < p.m && i0 + c < p.n) ? Elem<kT>::load(static_cast<const T *>(p.dy) + row * p.lddy + i0 + c) : 0.0f;
            float v = 0.0f;
            if (row < p.m && j0 + c < p.k)
                v = act2(both(decode8(static_cast<const uint8_t *>(p.x.q)[row * p.k + j0 + c], p.x.qkind) *
                              scale_at(p.x.scale, p.x.qmode, row, p.k, j0 + c)), act).x;
            xs[t][c] = v;
        }
        __syncthreads();
#pragma unroll
        for (int l = 0; l < 16; ++l) {
            if (tid < 64) sum += ds[l][tid];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ds[l][ty * 4 + i], xs[l][tx * 4 + j], acc[i][j]);
        }
        __syncthreads();
    }
    if (p.db && j0 == 0 && tid < 64 && i0 + tid < p.n) Elem<kT>::store(static_cast<T *>(p.db) + i0 + tid, sum);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = i0 + ty * 4 + i, c = j0 + tx * 4 + j;
            if (r < p.n && c < p.k) Elem<kT>::store(static_cast<T *>(p.dw) + r * p.k + c, acc[i][j]);
        }
}

template <class P>
cudaError_t launch(void (*kern)(P, Activation), int64_t tiles, const P &p, int act, cudaStream_t stream) {
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, activation_of(act));
    return e != cudaSuccess ? e : cudaGetLastError();
}

int64_t tiles64(int a, int b) { return ((a + 63ll) / 64) * ((b + 63ll) / 64); }

}  // namespace

cudaError_t launch_quant_product(bool bf16, const QuantProduct &p, cudaStream_t stream) {
    return launch(bf16 ? quant_product_any_kernel<ELEM_BF16> : quant_product_any_kernel<ELEM_F16>, tiles64(p.m, p.n), p, p.act, stream);
}

cudaError_t launch_quant_weight_grad(bool bf16, const QuantWeightGrad &p, cudaStream_t stream) {
    return launch(bf16 ? quant_weight_grad_any_kernel<ELEM_BF16> : quant_weight_grad_any_kernel<ELEM_F16>, tiles64(p.n, p.k), p, p.act,
                  stream);
}

}  // namespace mc2
