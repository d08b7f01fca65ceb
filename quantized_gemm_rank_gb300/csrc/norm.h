// norm.h -- the residual RMS norm's kernels, as the C entry points call them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mc2 {

// Strides are in elements, from row to row.
struct NormParams {
    const void *x, *res, *w;
    void *out, *res_out, *q, *scale;
    float *rstd;
    int64_t ldx, ldr, ldo, ldro;
    int64_t m;
    int h;
    float eps;
    int w_f32;   // the weight is fp32 (otherwise of x's type)
    int qmode, qkind;
};

struct NormGradParams {
    const void *dy, *x, *w, *dres;
    const float *rstd;
    void *dx, *dw;
    float *parts;   // norm_grad_parts() rows of h fp32 (with dw)
    int64_t lddy, ldx, lddres, lddx;
    int64_t m;
    int h;
    int w_f32;
};

// kind: ELEM_F16, ELEM_BF16 or ELEM_F32, the type of x and the outputs
cudaError_t launch_add_rms_norm(int kind, const NormParams &p, int num_sms, cudaStream_t stream);
// Shares of dw that the gradient's blocks leave in the workspace (more for 2-byte elements than for 4).
int norm_grad_parts(int64_t m, int64_t h, int elem_size);
cudaError_t launch_rms_norm_grad(int kind, const NormGradParams &p, cudaStream_t stream);
// dw from the shares that launch_rms_norm_grad left
cudaError_t launch_rms_norm_dw(int kind, const NormGradParams &p, cudaStream_t stream);

}  // namespace mc2
