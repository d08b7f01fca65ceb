// codes_api.cu -- the C entry points of the 8-bit path of a linear (the int8 product with scales per token and per
// channel, an activation kept in 8 bits, and its use in the backward pass): argument validation and stream-ordered launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include "host.h"
#include "kept.h"
#include "mc2_gb300.h"
#include "num.cuh"

namespace {

using namespace mc2::host;

constexpr int64_t kMostRows = 1ll << 30;   // of a matrix: its indices and a tile's past its end stay within 32 bits
constexpr int64_t kMostDepth = 131071;     // 2^14 times this many products of two int8 is below 2^31

int check_act(int act) {
    return act < MC2_ACT_NONE || act > MC2_ACT_SILU ? fail(MC2_ERR_DTYPE, "unknown activation %d", act) : MC2_OK;
}

int check_16bit(int dtype) {
    return dtype != MC2_F16 && dtype != MC2_BF16 ? fail(MC2_ERR_DTYPE, "dtype must be MC2_F16 or MC2_BF16 (got %d)", dtype) : MC2_OK;
}

int check_sizes(int64_t m, int64_t n, int64_t k) {
    if (m < 1 || n < 1 || k < 1)
        return fail(MC2_ERR_SHAPE, "empty tensors are not supported (m=%lld n=%lld k=%lld)", (long long)m, (long long)n, (long long)k);
    if (m > kMostRows || n > kMostRows || k > kMostRows) return fail(MC2_ERR_SHAPE, "m, n or k exceeds 2^30");
    return MC2_OK;
}

// The codes and scales of an activation that is kept.
int check_kept(const void *q, const void *scale, int64_t m, int64_t h, int quant_mode, int q_dtype, mc2::Kept *kept) {
    switch (quant_mode) {
        case MC2_QUANT_PERTOKEN_DYNAMIC: kept->qmode = mc2::QM_TOKEN; break;
        case MC2_QUANT_PERGROUP: kept->qmode = mc2::QM_GROUP; break;
        case MC2_QUANT_MX: kept->qmode = mc2::QM_MX; break;
        default: return fail(MC2_ERR_DTYPE, "quant_mode must be 4 (pergroup), 6 (mx) or 7 (pertoken dynamic), got %d", quant_mode);
    }
    if (q_dtype != MC2_I8 && q_dtype != MC2_F8E4M3 && q_dtype != MC2_F8E5M2)
        return fail(MC2_ERR_DTYPE, "q_dtype must be MC2_I8, MC2_F8E4M3 or MC2_F8E5M2 (got %d)", q_dtype);
    if (kept->qmode == mc2::QM_MX && q_dtype == MC2_I8)
        return fail(MC2_ERR_DTYPE, "mx scales need fp8 codes (MC2_F8E4M3 or MC2_F8E5M2)");
    if (int st = check_sizes(m, 1, h)) return st;
    if (!q || !scale) return fail(MC2_ERR_NULL, "q and scale are required");
    if (kept->qmode != mc2::QM_MX && reinterpret_cast<uintptr_t>(scale) % 4 != 0)
        return fail(MC2_ERR_UNSUPPORTED, "scale is not aligned to its 4-byte elements");
    kept->q = const_cast<void *>(q), kept->scale = const_cast<void *>(scale);
    kept->m = m, kept->h = static_cast<int>(h);
    kept->qkind = q_dtype == MC2_F8E4M3 ? mc2::Q_E4M3 : (q_dtype == MC2_F8E5M2 ? mc2::Q_E5M2 : mc2::Q_I8);
    return MC2_OK;
}

int check_any_dtype(int dtype) {
    return dtype != MC2_F16 && dtype != MC2_BF16 && dtype != MC2_F32
               ? fail(MC2_ERR_DTYPE, "dtype must be MC2_F16, MC2_BF16 or MC2_F32 (got %d)", dtype)
               : MC2_OK;
}

int check_workspace(const void *workspace, size_t given, size_t need) {
    if (need == 0) return MC2_OK;
    if (!workspace || given < need)
        return fail(MC2_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? given : (size_t)0);
    if (!aligned16(workspace)) return fail(MC2_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    return MC2_OK;
}

// The matrices of an int8 product.
int check_product(const int8_t *x, int64_t ldx, const int8_t *w, int64_t ldw, int w_is_nk, int64_t m, int64_t n, int64_t k,
                  const void *residual, int64_t ldr, const void *out, int64_t ldo, mc2::QuantProduct *p) {
    if (int st = check_sizes(m, n, k)) return st;
    if (k > kMostDepth) return fail(MC2_ERR_SHAPE, "k must be at most %lld, so that int32 holds any sum", (long long)kMostDepth);
    if (!x || !w || !out) return fail(MC2_ERR_NULL, "x, w and out are required");
    if (int st = check_rows("x", x, ldx, m, k, 1)) return st;
    if (int st = check_rows("w", w, ldw, w_is_nk ? n : k, w_is_nk ? k : n, 1)) return st;
    if (int st = check_rows("out", out, ldo, m, n, 2)) return st;
    if (residual) {
        if (int st = check_rows("residual", residual, ldr, m, n, 2)) return st;
        if (residual == out && m > 1 && ldr != ldo)
            return fail(MC2_ERR_SHAPE, "residual and out in one buffer need the same row stride");
    }
    p->x = x, p->w = w, p->residual = residual, p->out = const_cast<void *>(out);
    p->ldx = ldx, p->ldw = ldw, p->ldr = ldr, p->ldo = ldo;
    p->m = static_cast<int>(m), p->n = static_cast<int>(n), p->k = static_cast<int>(k);
    p->w_nk = w_is_nk != 0;
    return MC2_OK;
}

int check_weight_grad(const void *dy, int64_t lddy, const void *dw, int64_t m, int64_t n, int64_t k, mc2::QuantWeightGrad *p) {
    if (int st = check_sizes(m, n, k)) return st;
    if (!dy || !dw) return fail(MC2_ERR_NULL, "dy and dw are required");
    if (int st = check_rows("dy", dy, lddy, m, n, 2)) return st;
    if (int st = check_rows("dw", dw, k, n, k, 2)) return st;
    p->dy = dy, p->dw = const_cast<void *>(dw), p->lddy = lddy;
    p->m = static_cast<int>(m), p->n = static_cast<int>(n), p->k = static_cast<int>(k);
    return MC2_OK;
}

// Each kernel of a call of several is marked as it is launched.
void mark(void *marks) { static_cast<LaunchMarks *>(marks)->launched(); }

}  // namespace

extern "C" {

int mc2_quant_matmul_workspace(const int8_t *x, int64_t ldx, const int8_t *w, int64_t ldw, int w_is_nk, int64_t m, int64_t n,
                               int64_t k, const void *residual, int64_t ldr, const void *out, int64_t ldo, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(MC2_ERR_NULL, "bytes is NULL");
    mc2::QuantProduct p = {};
    if (int st = check_product(x, ldx, w, ldw, w_is_nk, m, n, k, residual, ldr, out, ldo, &p)) return st;
    *bytes = mc2::plan_quant_product(p).total;
    return MC2_OK;
}

int mc2_quant_matmul(const int8_t *x, int64_t ldx, const float *x_scale, const int8_t *w, int64_t ldw, int w_is_nk,
                     const float *w_scale, int64_t m, int64_t n, int64_t k, const void *bias, int bias_dtype, int act,
                     const void *residual, int64_t ldr, int dtype, void *out, int64_t ldo, void *workspace,
                     size_t workspace_bytes, void *stream) {
    clear_error();
    if (int st = check_16bit(dtype)) return st;
    if (int st = check_act(act)) return st;
    mc2::QuantProduct p = {};
    if (int st = check_product(x, ldx, w, ldw, w_is_nk, m, n, k, residual, ldr, out, ldo, &p)) return st;
    if (!x_scale || !w_scale) return fail(MC2_ERR_NULL, "x_scale and w_scale are required");
    if (int st = check_rows("x_scale", x_scale, m, 1, m, 4)) return st;
    if (int st = check_rows("w_scale", w_scale, n, 1, n, 4)) return st;
    if (bias) {
        if (bias_dtype != dtype && bias_dtype != MC2_F32)
            return fail(MC2_ERR_DTYPE, "the bias must be of the type of out or MC2_F32 (got %d)", bias_dtype);
        if (int st = check_rows("bias", bias, n, 1, n, elem_size(bias_dtype))) return st;
    }
    const mc2::ProductPlan plan = mc2::plan_quant_product(p);
    if (int st = check_workspace(workspace, workspace_bytes, plan.total)) return st;
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    p.x_scale = x_scale, p.w_scale = w_scale, p.bias = bias;
    p.act = act;
    p.bias_f32 = bias_dtype == MC2_F32;
    p.workspace = workspace;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_quant_product(dtype == MC2_BF16, p, plan, dev.num_sms, s, mark, &marks);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "quant_matmul launch: %s", cudaGetErrorString(e));
    return MC2_OK;
}

int mc2_act_quant(const void *z, int64_t ldz, int64_t m, int64_t h, int act, int dtype, int quant_mode, int q_dtype, void *q,
                  void *scale, void *stream) {
    clear_error();
    if (int st = check_any_dtype(dtype)) return st;
    if (int st = check_act(act)) return st;
    mc2::Kept kept = {};
    if (int st = check_kept(q, scale, m, h, quant_mode, q_dtype, &kept)) return st;
    if (!z) return fail(MC2_ERR_NULL, "z is required");
    if (int st = check_rows("z", z, ldz, m, h, elem_size(dtype))) return st;
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_act_quant(elem_kind(dtype), z, ldz, kept, act, dev.num_sms, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "act_quant launch: %s", cudaGetErrorString(e));
    marks.launched();
    return MC2_OK;
}

int mc2_act_dequant(const void *q, const void *scale, int64_t m, int64_t h, int act, int quant_mode, int q_dtype, int dtype,
                    void *out, int64_t ldo, void *stream) {
    clear_error();
    if (int st = check_any_dtype(dtype)) return st;
    if (int st = check_act(act)) return st;
    mc2::Kept kept = {};
    if (int st = check_kept(q, scale, m, h, quant_mode, q_dtype, &kept)) return st;
    if (!out) return fail(MC2_ERR_NULL, "out is required");
    if (int st = check_rows("out", out, ldo, m, h, elem_size(dtype))) return st;
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_act_dequant(elem_kind(dtype), kept, act, out, ldo, dev.num_sms, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "act_dequant launch: %s", cudaGetErrorString(e));
    marks.launched();
    return MC2_OK;
}

int mc2_act_grad_quant(const void *dy, int64_t lddy, const void *q, const void *scale, int64_t m, int64_t h, int act,
                       int quant_mode, int q_dtype, int dtype, void *dz, int64_t lddz, void *stream) {
    clear_error();
    if (int st = check_16bit(dtype)) return st;
    if (int st = check_act(act)) return st;
    mc2::Kept kept = {};
    if (int st = check_kept(q, scale, m, h, quant_mode, q_dtype, &kept)) return st;
    if (!dy || !dz) return fail(MC2_ERR_NULL, "dy and dz are required");
    if (int st = check_rows("dy", dy, lddy, m, h, 2)) return st;
    if (int st = check_rows("dz", dz, lddz, m, h, 2)) return st;
    if (dz == dy && m > 1 && lddz != lddy) return fail(MC2_ERR_SHAPE, "dy and dz in one buffer need the same row stride");
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_act_grad_quant(dtype == MC2_BF16, dy, lddy, kept, act, dz, lddz, dev.num_sms, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "act_grad_quant launch: %s", cudaGetErrorString(e));
    marks.launched();
    return MC2_OK;
}

int mc2_matmul_weight_grad_quant_workspace(const void *dy, int64_t lddy, const void *dw, int64_t m, int64_t n, int64_t k,
                                           size_t *bytes) {
    clear_error();
    if (!bytes) return fail(MC2_ERR_NULL, "bytes is NULL");
    mc2::QuantWeightGrad p = {};
    if (int st = check_weight_grad(dy, lddy, dw, m, n, k, &p)) return st;
    *bytes = mc2::quant_weight_grad_workspace(p);
    return MC2_OK;
}

int mc2_matmul_weight_grad_quant(const void *dy, int64_t lddy, const void *q, const void *scale, int64_t m, int64_t n, int64_t k,
                                 int act, int quant_mode, int q_dtype, int dtype, void *dw, void *db, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    clear_error();
    if (int st = check_16bit(dtype)) return st;
    if (int st = check_act(act)) return st;
    mc2::QuantWeightGrad p = {};
    if (int st = check_weight_grad(dy, lddy, dw, m, n, k, &p)) return st;
    if (int st = check_kept(q, scale, m, k, quant_mode, q_dtype, &p.x)) return st;
    if (db)
        if (int st = check_rows("db", db, n, 1, n, 2)) return st;
    if (int st = check_workspace(workspace, workspace_bytes, mc2::quant_weight_grad_workspace(p))) return st;
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    p.db = db, p.act = act, p.workspace = workspace;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_quant_weight_grad(dtype == MC2_BF16, p, dev.num_sms, s, mark, &marks);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "matmul_weight_grad_quant launch: %s", cudaGetErrorString(e));
    return MC2_OK;
}

}  // extern "C"
