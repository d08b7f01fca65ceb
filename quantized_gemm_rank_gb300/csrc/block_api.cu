// block_api.cu -- the C entry points of the operators around the fused linears
// (residual RMS norm and its gradient, the fused-epilogue matrix product and
// the activation gradients): argument validation and stream-ordered launches.
#include <cmath>
#include <cuda.h>
#include <cuda_runtime.h>

#include "host.h"
#include "linear.h"
#include "mc2_gb300.h"
#include "norm.h"
#include "num.cuh"

namespace {

using namespace mc2::host;

size_t elem_size(int dtype) { return dtype == MC2_F32 ? 4 : 2; }

int elem_kind(int dtype) {
    return dtype == MC2_F16 ? mc2::ELEM_F16 : (dtype == MC2_BF16 ? mc2::ELEM_BF16 : mc2::ELEM_F32);
}

// A matrix argument: its rows must not overlap and its elements must be aligned
// to their own size.  Optional ones are passed only when given.
int check_rows(const char *what, const void *p, int64_t ld, int64_t m, int64_t cols, size_t size) {
    if (ld < cols && m > 1)
        return fail(MC2_ERR_SHAPE, "%s: rows of %lld elements cannot be %lld elements apart", what, (long long)cols,
                    (long long)ld);
    if (ld > INT64_MAX / 4 / (m > 1 ? m : 1))
        return fail(MC2_ERR_SHAPE, "%s: a row stride of %lld elements is too large", what, (long long)ld);
    if (reinterpret_cast<uintptr_t>(p) % size != 0)
        return fail(MC2_ERR_UNSUPPORTED, "%s is not aligned to its %zu-byte elements", what, size);
    return MC2_OK;
}

int check_norm_sizes(int64_t m, int64_t h) {
    if (m < 1 || h < 1)
        return fail(MC2_ERR_SHAPE, "empty tensors are not supported (m=%lld h=%lld)", (long long)m, (long long)h);
    if (m > INT32_MAX || h > (1ll << 30)) return fail(MC2_ERR_SHAPE, "m exceeds INT32_MAX or h exceeds 2^30");
    return MC2_OK;
}

int check_norm_types(int dtype, int weight_dtype) {
    if (dtype != MC2_F16 && dtype != MC2_BF16 && dtype != MC2_F32)
        return fail(MC2_ERR_DTYPE, "dtype must be MC2_F16, MC2_BF16 or MC2_F32 (got %d)", dtype);
    if (weight_dtype != dtype && weight_dtype != MC2_F32)
        return fail(MC2_ERR_DTYPE, "the weight must be of the type of x or MC2_F32 (got %d)", weight_dtype);
    return MC2_OK;
}

int check_product(int64_t m, int64_t n, int64_t k, int act, int dtype) {
    if (dtype != MC2_F16 && dtype != MC2_BF16)
        return fail(MC2_ERR_DTYPE, "dtype must be MC2_F16 or MC2_BF16 (got %d)", dtype);
    if (act < MC2_ACT_NONE || act > MC2_ACT_SILU) return fail(MC2_ERR_DTYPE, "unknown activation %d", act);
    if (m < 1 || n < 1 || k < 1)
        return fail(MC2_ERR_SHAPE, "empty tensors are not supported (m=%lld n=%lld k=%lld)", (long long)m,
                    (long long)n, (long long)k);
    if (m > INT32_MAX || n > INT32_MAX || k > INT32_MAX) return fail(MC2_ERR_SHAPE, "m, n or k exceeds INT32_MAX");
    return MC2_OK;
}

// The product itself, its arguments checked: the kernel that takes its sizes and layout.
int product(const char *what, bool bf16, mc2::LinearParams &p, void *stream) {
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the stride of a single row is free: one that the tensor copies take
    const auto one_row = [](int rows, int64_t cols, int64_t &ld) {
        if (rows == 1) ld = (cols + 7) / 8 * 8;
    };
    one_row(p.m, p.k, p.ldx);
    one_row(p.w_nk ? p.n : p.k, p.w_nk ? p.k : p.n, p.ldw);
    one_row(p.m, p.n, p.ldo);
    one_row(p.m, p.n, p.ldp);
    one_row(p.m, p.n, p.ldaux);
    LaunchMarks marks(s);
    cudaError_t e = !mc2::linear_layout_fits(p) ? mc2::launch_linear_any(bf16, p, s)
                    : mc2::linear_prefers_split(p, dev.num_sms)
                        ? mc2::launch_linear_split(bf16, p, dev.num_sms, s)
                        : mc2::launch_linear_tiles(bf16, p, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    marks.launched();
    return MC2_OK;
}

}  // namespace

extern "C" {

int mc2_add_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                     int weight_dtype, int64_t m, int64_t h, float eps, int dtype, void *out, int64_t ldo,
                     void *residual_out, int64_t ldro, float *rstd_out, int quant_mode, int q_dtype, void *q_out,
                     void *scale_out, void *stream) {
    clear_error();
    if (int st = check_norm_types(dtype, weight_dtype)) return st;
    if (int st = check_norm_sizes(m, h)) return st;
    if (!x || !weight) return fail(MC2_ERR_NULL, "x and weight are required");
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(MC2_ERR_SHAPE, "eps must be finite and at least 0");
    int qmode = mc2::QM_NONE;
    switch (quant_mode) {
        case MC2_QUANT_NONE: break;
        case MC2_QUANT_PERTOKEN_DYNAMIC: qmode = mc2::QM_TOKEN; break;
        case MC2_QUANT_PERGROUP: qmode = mc2::QM_GROUP; break;
        case MC2_QUANT_MX: qmode = mc2::QM_MX; break;
        default:
            return fail(MC2_ERR_DTYPE, "quant_mode must be 0 (none), 4 (pergroup), 6 (mx) or 7 (pertoken dynamic), got %d",
                        quant_mode);
    }
    if (qmode == mc2::QM_NONE) {
        if (!out) return fail(MC2_ERR_NULL, "out is required without a quantised output");
        if (q_out || scale_out) return fail(MC2_ERR_SHAPE, "q_out and scale_out must be NULL when quant_mode is 0");
    } else {
        if (!q_out || !scale_out) return fail(MC2_ERR_NULL, "quant_mode %d needs q_out and scale_out", quant_mode);
        if (q_dtype != MC2_I8 && q_dtype != MC2_F8E4M3 && q_dtype != MC2_F8E5M2)
            return fail(MC2_ERR_DTYPE, "q_dtype must be MC2_I8, MC2_F8E4M3 or MC2_F8E5M2 (got %d)", q_dtype);
        if (qmode == mc2::QM_MX && q_dtype == MC2_I8)
            return fail(MC2_ERR_DTYPE, "mx scales need fp8 codes (MC2_F8E4M3 or MC2_F8E5M2)");
        if (qmode != mc2::QM_MX && reinterpret_cast<uintptr_t>(scale_out) % 4 != 0)
            return fail(MC2_ERR_UNSUPPORTED, "scale_out is not aligned to its 4-byte elements");
    }
    if (residual_out && !residual) return fail(MC2_ERR_SHAPE, "residual_out must be NULL without a residual");
    if (residual_out && residual_out == out) return fail(MC2_ERR_SHAPE, "residual_out and out must be two buffers");
    const size_t es = elem_size(dtype);
    if (int st = check_rows("x", x, ldx, m, h, es)) return st;
    if (residual)
        if (int st = check_rows("residual", residual, ldr, m, h, es)) return st;
    if (out)
        if (int st = check_rows("out", out, ldo, m, h, es)) return st;
    if (residual_out)
        if (int st = check_rows("residual_out", residual_out, ldro, m, h, es)) return st;
    if (int st = check_rows("weight", weight, h, 1, h, elem_size(weight_dtype))) return st;
    if (rstd_out && reinterpret_cast<uintptr_t>(rstd_out) % 4 != 0)
        return fail(MC2_ERR_UNSUPPORTED, "rstd_out is not aligned to its 4-byte elements");

    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    mc2::NormParams p = {};
    p.x = x, p.res = residual, p.w = weight;
    p.out = out, p.res_out = residual_out, p.q = q_out, p.scale = scale_out, p.rstd = rstd_out;
    p.ldx = ldx, p.ldr = ldr, p.ldo = ldo, p.ldro = ldro;
    p.m = m, p.h = static_cast<int>(h), p.eps = eps;
    p.w_f32 = weight_dtype == MC2_F32;
    p.qmode = qmode;
    p.qkind = q_dtype == MC2_F8E4M3 ? mc2::Q_E4M3 : (q_dtype == MC2_F8E5M2 ? mc2::Q_E5M2 : mc2::Q_I8);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_add_rms_norm(elem_kind(dtype), p, dev.num_sms, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "RMS norm launch: %s", cudaGetErrorString(e));
    marks.launched();
    return MC2_OK;
}

int mc2_rms_norm_grad_workspace(int64_t m, int64_t h, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(MC2_ERR_NULL, "bytes is NULL");
    if (int st = check_norm_sizes(m, h)) return st;
    *bytes = static_cast<size_t>(mc2::norm_grad_parts(m, h, 2)) * static_cast<size_t>(h) * 4;
    return MC2_OK;
}

int mc2_rms_norm_grad(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *weight, int weight_dtype,
                      const float *rstd, const void *dres, int64_t lddres, int64_t m, int64_t h, int dtype, void *dx,
                      int64_t lddx, void *dw, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    if (int st = check_norm_types(dtype, weight_dtype)) return st;
    size_t need = 0;
    if (int st = mc2_rms_norm_grad_workspace(m, h, &need)) return st;
    if (!dy || !x || !weight || !rstd || !dx) return fail(MC2_ERR_NULL, "dy, x, weight, rstd and dx are required");
    const size_t es = elem_size(dtype);
    if (int st = check_rows("dy", dy, lddy, m, h, es)) return st;
    if (int st = check_rows("x", x, ldx, m, h, es)) return st;
    if (int st = check_rows("dx", dx, lddx, m, h, es)) return st;
    if (dres)
        if (int st = check_rows("dres", dres, lddres, m, h, es)) return st;
    if (int st = check_rows("weight", weight, h, 1, h, elem_size(weight_dtype))) return st;
    if (int st = check_rows("rstd", rstd, m, 1, m, 4)) return st;
    if (dw) {
        if (int st = check_rows("dw", dw, h, 1, h, elem_size(weight_dtype))) return st;
        if (!workspace || workspace_bytes < need)
            return fail(MC2_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                        workspace ? workspace_bytes : (size_t)0);
        if (!aligned16(workspace)) return fail(MC2_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    }

    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    mc2::NormGradParams p = {};
    p.dy = dy, p.x = x, p.w = weight, p.dres = dres, p.rstd = rstd, p.dx = dx, p.dw = dw;
    p.parts = static_cast<float *>(workspace);
    p.lddy = lddy, p.ldx = ldx, p.lddres = lddres, p.lddx = lddx;
    p.m = m, p.h = static_cast<int>(h);
    p.w_f32 = weight_dtype == MC2_F32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_rms_norm_grad(elem_kind(dtype), p, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "RMS norm gradient launch: %s", cudaGetErrorString(e));
    marks.launched();
    if (dw) {
        e = mc2::launch_rms_norm_dw(elem_kind(dtype), p, s);
        if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "RMS norm weight gradient launch: %s", cudaGetErrorString(e));
        marks.launched();
    }
    return MC2_OK;
}

int mc2_matmul_bias_act(const void *x, int64_t ldx, const void *w, int64_t ldw, int w_is_nk, int64_t m, int64_t n,
                        int64_t k, const void *bias, int act, const void *residual, int64_t ldr, int dtype, void *out,
                        int64_t ldo, void *preact, int64_t ldp, void *stream) {
    clear_error();
    if (int st = check_product(m, n, k, act, dtype)) return st;
    if (!x || !w || !out) return fail(MC2_ERR_NULL, "x, w and out are required");
    if (int st = check_rows("x", x, ldx, m, k, 2)) return st;
    if (int st = check_rows("w", w, ldw, w_is_nk ? n : k, w_is_nk ? k : n, 2)) return st;
    if (int st = check_rows("out", out, ldo, m, n, 2)) return st;
    if (bias)
        if (int st = check_rows("bias", bias, n, 1, n, 2)) return st;
    if (residual)
        if (int st = check_rows("residual", residual, ldr, m, n, 2)) return st;
    if (preact) {
        if (int st = check_rows("preact", preact, ldp, m, n, 2)) return st;
        if (preact == out || preact == residual)
            return fail(MC2_ERR_SHAPE, "preact must be a buffer of its own");
    }
    mc2::LinearParams p = {};
    p.x = x, p.w = w, p.bias = bias, p.aux = residual, p.out = out, p.preact = preact;
    p.ldx = ldx, p.ldw = ldw, p.ldaux = ldr, p.ldo = ldo, p.ldp = ldp;
    p.m = static_cast<int>(m), p.n = static_cast<int>(n), p.k = static_cast<int>(k);
    p.w_nk = w_is_nk != 0;
    p.act = act;
    p.aux_mode = residual ? mc2::AUX_RESIDUAL : mc2::AUX_NONE;
    return product("matmul_bias_act", dtype == MC2_BF16, p, stream);
}

int mc2_matmul_act_grad(const void *dy, int64_t lddy, const void *w, int64_t ldw, int w_is_nk, const void *z,
                        int64_t ldz, int act, int64_t m, int64_t n, int64_t k, int dtype, void *dz, int64_t lddz,
                        void *stream) {
    clear_error();
    if (int st = check_product(m, n, k, act, dtype)) return st;
    if (!dy || !w || !z || !dz) return fail(MC2_ERR_NULL, "dy, w, z and dz are required");
    if (int st = check_rows("dy", dy, lddy, m, n, 2)) return st;
    if (int st = check_rows("w", w, ldw, w_is_nk ? n : k, w_is_nk ? k : n, 2)) return st;
    if (int st = check_rows("z", z, ldz, m, k, 2)) return st;
    if (int st = check_rows("dz", dz, lddz, m, k, 2)) return st;
    // the product's own sizes: (m, k) out of a contraction over n, with the
    // forward weight (n, k) as a (contraction, columns) operand
    mc2::LinearParams p = {};
    p.x = dy, p.w = w, p.aux = z, p.out = dz;
    p.ldx = lddy, p.ldw = ldw, p.ldaux = ldz, p.ldo = lddz;
    p.m = static_cast<int>(m), p.n = static_cast<int>(k), p.k = static_cast<int>(n);
    p.w_nk = w_is_nk == 0;
    p.act = act;
    p.aux_mode = mc2::AUX_ACT_GRAD;
    return product("matmul_act_grad", dtype == MC2_BF16, p, stream);
}

int mc2_act_grad(const void *dy, int64_t lddy, const void *z, int64_t ldz, int act, int64_t m, int64_t n, int dtype,
                 void *dz, int64_t lddz, void *stream) {
    clear_error();
    if (int st = check_product(m, n, 1, act, dtype)) return st;
    if (!dy || !z || !dz) return fail(MC2_ERR_NULL, "dy, z and dz are required");
    if (int st = check_rows("dy", dy, lddy, m, n, 2)) return st;
    if (int st = check_rows("z", z, ldz, m, n, 2)) return st;
    if (int st = check_rows("dz", dz, lddz, m, n, 2)) return st;
    DeviceInfo dev;
    if (int st = current_device(&dev)) return st;
    const mc2::ActGradParams p = {dy, z, dz, lddy, ldz, lddz, m, n, act};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchMarks marks(s);
    cudaError_t e = mc2::launch_act_grad(dtype == MC2_BF16, p, dev.num_sms, s);
    if (e != cudaSuccess) return fail(MC2_ERR_CUDA, "act_grad launch: %s", cudaGetErrorString(e));
    marks.launched();
    return MC2_OK;
}

}  // extern "C"
