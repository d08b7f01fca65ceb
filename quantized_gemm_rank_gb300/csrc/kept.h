// kept.h -- an activation kept in 8 bits, and its uses: the kernels, as the C entry points call them.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mc2 {

// Codes (m, h) without gaps, and their scales: fp32 per row (QM_TOKEN) or per 128 columns (QM_GROUP), or e8m0 codes
// per 32 columns (QM_MX).
struct Kept {
    void *q, *scale;
    int64_t m;
    int h;
    int qmode, qkind;
};

// codes of act(z); z of elem kind (rows ldz apart)
cudaError_t launch_act_quant(int kind, const void *z, int64_t ldz, const Kept &to, int act, int num_sms, cudaStream_t stream);
// out = act(q scale), of elem kind
cudaError_t launch_act_dequant(int kind, const Kept &from, int act, void *out, int64_t ldo, int num_sms, cudaStream_t stream);
// dz = dy act'(q scale), 16-bit
cudaError_t launch_act_grad_quant(bool bf16, const void *dy, int64_t lddy, const Kept &z, int act, void *dz, int64_t lddz,
                                  int num_sms, cudaStream_t stream);

// out (m, n) = act(float(x w^T) x_scale w_scale + bias) + residual; x (m, k) and w int8, w (n, k) or (k, n) (w_nk == 0)
struct QuantProduct {
    const int8_t *x, *w;
    const float *x_scale, *w_scale;
    const void *bias, *residual;
    void *out;
    int64_t ldx, ldw, ldr, ldo;
    int m, n, k;
    int w_nk;
    int act;
    int bias_f32;   // (otherwise of out's type)
    void *workspace;
};
// One to eight tokens and an (n, k) weight, in any layout.
cudaError_t launch_quant_tokens(bool bf16, const QuantProduct &p, cudaStream_t stream);
// How a product is computed, and the pieces of its workspace (in bytes from its start).
struct ProductPlan {
    size_t x = 0, w = 0, out = 0, total = 0;
    bool tokens = false;       // the kernel of one to eight tokens, on the matrices as they are
    bool split = false;        // the one of few tokens, on int8 operands
    bool x_apart = false, w_apart = false;   // the operands go through the workspace (the tiles': always)
    bool out_apart = false;    // the output, too
    bool residual_in = false;  // the residual is copied to where the output will be
};
ProductPlan plan_quant_product(const QuantProduct &p);   // by the matrices and sizes
// Kernels of a call, each followed by mark(ctx)
using Mark = void (*)(void *ctx);
cudaError_t launch_quant_product(bool bf16, const QuantProduct &p, const ProductPlan &at, int num_sms, cudaStream_t stream, Mark mark, void *ctx);

// dw (n, k) = dy^T act(q scale), db (n) = column sums of dy (or none); x is (m, k)
struct QuantWeightGrad {
    const void *dy;
    void *dw, *db;
    Kept x;
    int64_t lddy;
    int m, n, k;
    int act;
    void *workspace;
};
size_t quant_weight_grad_workspace(const QuantWeightGrad &p);
cudaError_t launch_quant_weight_grad(bool bf16, const QuantWeightGrad &p, int num_sms, cudaStream_t stream, Mark mark, void *ctx);

}  // namespace mc2
