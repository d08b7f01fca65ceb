// linear_tiles.cu -- the fused-epilogue matrix product of many rows: the GEMM of
// gemm_tcgen05.cuh with its tiles taken at run time and the epilogue forms of
// epilogue.cuh.  The epilogue reads a tile's sums from TMEM where it uses them; those of a
// contraction of several K blocks (see linear_tiles_block) are added in registers and put back there first
// (4096 to 8192 deep this takes 1% more than one accumulator over all of it).
// The tensor pipe bounds it, and called in turn the power limit: 8192 x 8192 x 7168 with bias, gelu and the
// pre-activation 520 us (1852 TFLOP/s) in a graph of a few launches, 597 to 610 us in turn; without an
// epilogue 493 in the graph.  Two more forms: int8 codes held as fp16, whose blocks of 1024 are added as integers and scaled
// by row and column (2048 tokens, 4096 x 4096: 41 us), and the parts of a weight gradient's sums in fp32.
#include "gemm_tcgen05.cuh"
#include "host.h"
#include "internal.h"
#include "linear.h"

namespace mc2 {

namespace {

template <bool kBF16, int kEpi>
cudaError_t launch_tiles(GemmParams &p, cudaStream_t stream) {
    using Cfg = TileCfg<2, true>;
    auto kern = mc2_gemm_kernel<2, kBF16, false, false, true, false, kEpi>;
    thread_local unsigned long long ready_ctx = 0;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ctx != ready_ctx) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
        if (e != cudaSuccess) return e;
        ready_ctx = ctx;
    }
    const int64_t tiles = ((p.m + Cfg::kTileM - 1ll) / Cfg::kTileM) * ((p.n + kBN - 1ll) / kBN) * (kEpi == EPI_SUMS ? p.splits : 1);
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * tiles), 1, 1);
    cfg.blockDim = dim3(kNumThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_tiles(bool bf16, const LinearParams &lp, cudaStream_t stream) {
    GemmParams p = {};
    const uint64_t m = lp.m, n = lp.n, k = lp.k;
    bool ok = host::make_map16(&p.a_maps[0], lp.x, k, m, kBK, kBM, lp.ldx);
    if (lp.w_nk) {
        ok = ok && host::make_map16(&p.b_map, lp.w, k, n, kBK, kBN / 2, lp.ldw);
    } else {
        p.b_mn_major = 1;
        if (host::make_map16_nmajor3d(&p.b_map, lp.w, n, k, kBK, kBN / 2 / 64, lp.ldw))
            p.b_3d = 1;
        else
            ok = ok && host::make_map16(&p.b_map, lp.w, n, k, 64, kBK, lp.ldw);
    }
    ok = ok && host::make_map16(&p.out_map, lp.out, n, m, 32, 32, lp.ldo);
    if (lp.aux_mode != AUX_NONE) {
        p.has_aux = 1;
        ok = ok && host::make_map16(&p.aux_map, lp.aux, n, m, 32, 32, lp.ldaux);
    }
    if (lp.preact) {
        p.has_pre = 1;
        ok = ok && host::make_map16(&p.pre_map, lp.preact, n, m, 32, 32, lp.ldp);
    }
    if (!ok) return cudaErrorInvalidValue;
    p.num_a_maps = 1;
    p.a_mode = A_SINGLE;
    p.m = lp.m, p.n = lp.n, p.k = lp.k;
    p.out = lp.out;
    p.act = activation_of(lp.act);
    p.wait_limit_ns = host::kWaitLimitNs;
    p.status = device_status_word();
    if (lp.codes) {
        p.kblock_tiles = 1024 / kBK;   // (an fp32 accumulator holds the sum of 1024 products of two int8 exactly)
        p.x1_scale = lp.x_scale, p.x2_scale = lp.w_scale;
        if (lp.bias_f32)
            p.bias_f32 = static_cast<const float *>(lp.bias);
        else
            p.bias16 = lp.bias;
        return bf16 ? launch_tiles<true, EPI_SCALED>(p, stream) : launch_tiles<false, EPI_SCALED>(p, stream);
    }
    p.kblock_tiles = linear_tiles_block(lp.k);
    p.bias16 = lp.bias;
    if (lp.aux_mode == AUX_ACT_GRAD)
        return bf16 ? launch_tiles<true, EPI_BACKWARD>(p, stream) : launch_tiles<false, EPI_BACKWARD>(p, stream);
    return bf16 ? launch_tiles<true, EPI_FORWARD>(p, stream) : launch_tiles<false, EPI_FORWARD>(p, stream);
}

cudaError_t launch_weight_grad_parts(bool bf16, const WeightGradParts &w, cudaStream_t stream) {
    GemmParams p = {};
    bool ok = true;
    if (host::make_map16_nmajor3d(&p.a_maps[0], w.dy, w.n, w.m, kBK, kBM / 64, w.lddy))
        p.a_3d = 1;
    else
        ok = host::make_map16(&p.a_maps[0], w.dy, w.n, w.m, 64, kBK, w.lddy);
    if (host::make_map16_nmajor3d(&p.b_map, w.x, w.k, w.m, kBK, kBN / 2 / 64, w.ldx))
        p.b_3d = 1;
    else
        ok = ok && host::make_map16(&p.b_map, w.x, w.k, w.m, 64, kBK, w.ldx);
    ok = ok && host::make_map32_parts(&p.out_map, w.parts, w.k, w.n, w.splits, w.ldp);
    if (!ok) return cudaErrorInvalidValue;
    p.num_a_maps = 1;
    p.a_mode = A_SINGLE_MN;
    p.b_mn_major = 1;
    p.m = w.n, p.n = w.k, p.k = w.m;
    p.kblock_tiles = w.block_tiles;
    p.splits = w.splits, p.split_blocks = w.split_blocks;
    p.colsum_out = w.col_parts;
    p.col_share = 1;
    p.wait_limit_ns = host::kWaitLimitNs;
    p.status = device_status_word();
    return bf16 ? launch_tiles<true, EPI_SUMS>(p, stream) : launch_tiles<false, EPI_SUMS>(p, stream);
}

}  // namespace mc2
