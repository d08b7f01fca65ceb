// linear_split.cu -- the fused-epilogue matrix product when there are few tiles:
// few rows (a decode step, a short chunk) or a small output.
//
// What bounds it is reading the weight once, so every SM has to read.  The
// weight's columns are the MMA's 128 rows and the tokens its N columns (16 to
// 256), so a single token wastes a 16-wide MMA and no weight traffic; the
// contraction is split over the CTAs of a cluster, whose partial sums are added
// in shared memory, in rank order (the result does not depend on timing).
//   warp 0      TMA producer (one lane)
//   warp 1      TMEM allocation, MMA issue
//   warps 4-7   partial sums from TMEM to shared memory
//   all warps   the sum over the cluster, and the epilogue, eight columns a thread
// The tensor core adds at the size of its running sum, so each 1024-deep part of
// the contraction goes to an accumulator of its own while TMEM has room, and
// these are added in fp32 with round-to-nearest.
#include "epilogue.cuh"
#include "host.h"
#include "internal.h"
#include "linear.h"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kTileN = 128;      // weight columns a tile (MMA M)
constexpr int kDepth = 64;       // contraction a stage
constexpr int kMaxStages = 16;
constexpr int kMaxCluster = 8;
constexpr int kSplitThreads = 256;
constexpr int kBlockSteps = 1024 / kDepth;   // stages of one accumulator
constexpr uint32_t kWBytes = kTileN * kDepth * 2;
constexpr uint32_t kSmemPerSm = 228 * 1024;
constexpr uint32_t kSmemStatic = 272;            // this kernel's static shared memory
constexpr uint32_t kSmemOverhead = 1024 + kSmemStatic;   // with the system's part of each CTA's

struct SplitParams {
    CUtensorMap w_map, x_map;
    const void *bias, *aux;
    void *out, *preact;
    int64_t ldaux, ldo, ldp;
    int m, n, steps;          // steps: 64-deep stages of the whole contraction
    int w_kn;                 // the weight is (k, n): read M-major
    int rows;                 // tokens a tile (MMA N), a multiple of 16
    int m_tiles, split;       // token tiles; CTAs a cluster
    int stages, accs, tmem_cols;
    int aligned;              // out, aux and preact rows are 16-byte aligned
    Activation act;
    int *status;
    uint64_t wait_limit_ns;
};

// A float4 of a CTA of this cluster (shared::cluster address).
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <bool kBF16>
__device__ __forceinline__ void store8(void *base, int64_t row_off, int col, int n, bool aligned, const float (&v)[8]) {
    uint16_t *p = static_cast<uint16_t *>(base) + row_off + col;
    uint32_t pk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pk[i] = pack2<kBF16>(v[2 * i], v[2 * i + 1]);
    if (aligned && col + 8 <= n) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < n) p[i] = static_cast<uint16_t>(pk[i >> 1] >> ((i & 1) * 16));
    }
}

__device__ __forceinline__ uint4 load8(const void *base, int64_t row_off, int col, int n, bool aligned) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + row_off + col;
    if (aligned && col + 8 <= n) return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << ((i & 1) * 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kBF16, int kEpi>
__global__ void __launch_bounds__(kSplitThreads, 1) linear_split_kernel(const __grid_constant__ SplitParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.stages;
    const uint32_t stage_bytes = kWBytes + static_cast<uint32_t>(p.rows) * kDepth * 2;
    const int rank = p.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    const int tile = blockIdx.x / p.split;
    const int n0 = tile / p.m_tiles * kTileN;            // clusters next to one another share the weight's tile
    const int m0 = tile % p.m_tiles * p.rows;
    const int step0 = static_cast<int>(static_cast<int64_t>(p.steps) * rank / p.split);
    const int count = static_cast<int>(static_cast<int64_t>(p.steps) * (rank + 1) / p.split) - step0;

    if (threadIdx.x == 0) {
        failed = 0;
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(ptx::smem_u32(&full_bar[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&empty_bar[s]), 1);
        }
        ptx::mbar_init(ptx::smem_u32(&done_bar), 1);
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc<1>(ptx::smem_u32(&tmem_slot), static_cast<uint32_t>(p.tmem_cols));
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&p.w_map);
        ptx::prefetch_tmap(&p.x_map);
        int stage = 0, issued = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            const uint32_t full = ptx::smem_u32(&full_bar[stage]);
            if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), phase, p.wait_limit_ns)) {
                ok = false;
                break;
            }
            const uint32_t sw = ptx::smem_u32(smem) + stage * stage_bytes;
            const int k0 = (step0 + i) * kDepth;
            ptx::mbar_arrive_expect_tx(full, stage_bytes);
            if (p.w_kn) {
                ptx::tma_load_2d(sw, &p.w_map, n0, k0, full);
                ptx::tma_load_2d(sw + kWBytes / 2, &p.w_map, n0 + 64, k0, full);
            } else {
                ptx::tma_load_2d(sw, &p.w_map, k0, n0, full);
            }
            ptx::tma_load_2d(sw + kWBytes, &p.x_map, k0, m0, full);
            ++issued;
            if (++stage == S) stage = 0, phase ^= 1u;
        }
        if (!ok) {
            atomicExch(&failed, 1);
            // the copies in flight land before the CTA can exit
            for (int back = 1; back <= S && back <= issued; ++back) {
                const int i = issued - back;
                (void)ptx::mbar_wait(ptx::smem_u32(&full_bar[i % S]), static_cast<uint32_t>((i / S) & 1), p.wait_limit_ns);
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_f16(kBF16, false, kTileN, p.rows, p.w_kn != 0);
        const uint32_t s0 = ptx::smem_u32(smem);
        const uint64_t w_desc0 = p.w_kn ? ptx::smem_desc_sw128(s0, kDepth * 128, 1024) : ptx::smem_desc_sw128(s0, 16, 1024);
        const uint64_t x_desc0 = ptx::smem_desc_sw128(s0 + kWBytes, 16, 1024);
        const uint32_t w_kk = p.w_kn ? (2048u >> 4) : (32u >> 4);
        const uint32_t x_kk = 32u >> 4;
        int stage = 0, in_block = 0, acc = 0, blocks = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            const bool got = ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), phase, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(stage) * (stage_bytes >> 4);
            const uint32_t d = tmem + static_cast<uint32_t>(acc * p.rows);
            // an accumulator's first stage starts it from zero
            ptx::mma_f16_ss<1>(d, w_desc0 + off, x_desc0 + off, idesc, in_block > 0 || blocks >= p.accs ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < kDepth / 16; ++kk)
                ptx::mma_f16_ss<1>(d, w_desc0 + off + kk * w_kk, x_desc0 + off + kk * x_kk, idesc, 1u);
            ptx::mma_commit<1>(ptx::smem_u32(&empty_bar[stage]));
            if (++stage == S) stage = 0, phase ^= 1u;
            if (++in_block == kBlockSteps) {
                in_block = 0;
                ++blocks;
                if (++acc == p.accs) acc = 0;
            }
        }
        if (!ok && lane == 0) atomicExch(&failed, 1);
        // (also after giving up: the MMAs issued so far complete before TMEM is freed)
        ptx::mma_commit_local<1>(ptx::smem_u32(&done_bar));
    }
    __syncwarp();
    // every thread waits (bounded) for the MMAs: from here on the ring is idle
    if (!ptx::mbar_wait(ptx::smem_u32(&done_bar), 0u, p.wait_limit_ns)) atomicExch(&failed, 1);
    __syncthreads();
    const bool ok = failed == 0;
    float *part = reinterpret_cast<float *>(smem);   // [rows][128], over the ring
    if (warp >= 4 && ok) {
        ptx::tc_fence_after();
        const int q = warp & 3;
        const int used = min(p.accs, (count + kBlockSteps - 1) / kBlockSteps);
        for (int c = 0; c < p.rows; c += 16) {
            float sum[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
            for (int a = 0; a < used; ++a) {
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * q) << 16) + a * p.rows + c, r);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] = __fadd_rn(sum[i], __uint_as_float(r[i]));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * kTileN + 32 * q + lane] = sum[i];
        }
        ptx::tc_fence_before();
    }
    if (!ok && threadIdx.x == 0 && p.status) atomicExch(p.status, -7);
    __syncwarp();
    if (p.split > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    // this CTA's share of the tile's tokens, the partial sums of all CTAs in rank order
    const int t0 = p.rows * rank / p.split, t1 = p.rows * (rank + 1) / p.split;
    const uint32_t part0 = ptx::smem_u32(part);
    for (int e = t0 * 16 + static_cast<int>(threadIdx.x); e < t1 * 16 && ok; e += kSplitThreads) {
        const int t = e >> 4, col = n0 + (e & 15) * 8;
        const int row = m0 + t;
        if (row >= p.m || col >= p.n) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        const uint32_t at = part0 + static_cast<uint32_t>(e) * 32u;
        for (int r = 0; r < p.split; ++r) {
            const uint32_t a = p.split > 1 ? ptx::mapa(at, r) : at;
            const float4 lo = load_cluster4(a), hi = load_cluster4(a + 16);
            v[0] = __fadd_rn(v[0], lo.x), v[1] = __fadd_rn(v[1], lo.y), v[2] = __fadd_rn(v[2], lo.z), v[3] = __fadd_rn(v[3], lo.w);
            v[4] = __fadd_rn(v[4], hi.x), v[5] = __fadd_rn(v[5], hi.y), v[6] = __fadd_rn(v[6], hi.z), v[7] = __fadd_rn(v[7], hi.w);
        }
        if (p.bias) {
            float b[8];
            load_bias8<kBF16>(p.bias, col, p.n, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], b[i]);
        }
        const bool vec = p.aligned != 0;
        if (p.preact) store8<kBF16>(p.preact, row * p.ldp, col, p.n, vec, v);
        uint4 a[1] = {make_uint4(0, 0, 0, 0)};
        if (p.aux) a[0] = load8(p.aux, row * p.ldaux, col, p.n, vec);
        epilogue<kBF16, kEpi>(v, a, p.act, p.aux != nullptr);
        store8<kBF16>(p.out, row * p.ldo, col, p.n, vec, v);
    }
    __syncwarp();
    if (p.split > 1)
        ptx::cluster_sync();   // no CTA leaves while another reads its sums
    else
        __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<1>(tmem, static_cast<uint32_t>(p.tmem_cols));
    }
}

// The shape of a launch for one number of tokens a tile.
struct SplitShape {
    int rows, m_tiles, split, stages, accs, tmem_cols, per_sm;
    uint32_t smem;
    int64_t tiles;
};

SplitShape split_shape(const LinearParams &p, int num_sms) {
    SplitShape s = {};
    s.rows = p.m <= 16 ? 16 : (p.m <= 32 ? 32 : (p.m <= 64 ? 64 : (p.m <= 128 ? 128 : 256)));
    s.m_tiles = (p.m + s.rows - 1) / s.rows;
    s.tiles = static_cast<int64_t>(s.m_tiles) * ((p.n + kTileN - 1) / kTileN);
    const int steps = (p.k + kDepth - 1) / kDepth;
    // short stages leave room for two CTAs an SM (and half of TMEM each)
    s.per_sm = s.rows <= 64 ? 2 : 1;
    const int64_t slots = static_cast<int64_t>(num_sms) * s.per_sm;
    int split = static_cast<int>(slots / s.tiles);
    if (split > kMaxCluster) split = kMaxCluster;
    if (split > steps) split = steps;
    if (split < 1) split = 1;
    s.split = split;
    const int most = (steps + split - 1) / split;   // stages of one CTA
    const uint32_t stage = kWBytes + static_cast<uint32_t>(s.rows) * kDepth * 2;
    const uint32_t room = s.per_sm == 2 ? 110u * 1024u : 220u * 1024u;
    s.stages = static_cast<int>(room / stage);
    if (s.stages > kMaxStages) s.stages = kMaxStages;
    if (s.stages > most) s.stages = most;
    uint32_t bytes = s.stages * stage;
    const uint32_t sums = static_cast<uint32_t>(s.rows) * kTileN * 4;
    if (bytes < sums) bytes = sums;
    s.smem = bytes + 1024;   // (slack to align the ring)
    const int blocks = (most + kBlockSteps - 1) / kBlockSteps;
    const int cols = s.per_sm == 2 ? 256 : 512;
    s.accs = cols / s.rows;
    if (s.accs > blocks) s.accs = blocks;
    s.tmem_cols = 32;
    while (s.tmem_cols < s.accs * s.rows) s.tmem_cols *= 2;
    // A CTA that waits for TMEM while its cluster's others hold theirs could wait for
    // ever on a CTA that waits for it, were TMEM oversubscribed by launches of two
    // streams.  So a CTA that takes 1/2^i of TMEM takes at least that part of the
    // SM's shared memory too (its static part and the system's 1 KiB included):
    // CTAs that fit beside one another find their columns free.
    const uint32_t share = static_cast<uint32_t>(s.tmem_cols) * (kSmemPerSm / 512) - kSmemOverhead;
    if (s.smem < share) s.smem = share;
    return s;
}

template <bool kBF16, int kEpi>
cudaError_t launch_split(const SplitParams &p, const SplitShape &s, cudaStream_t stream) {
    auto kern = linear_split_kernel<kBF16, kEpi>;
    thread_local unsigned long long ready_ctx = 0;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ctx != ready_ctx) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             227 * 1024 - kSmemStatic);
        if (e != cudaSuccess) return e;
        ready_ctx = ctx;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(s.tiles * s.split), 1, 1);
    cfg.blockDim = dim3(kSplitThreads, 1, 1);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = s.split > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

bool rows_aligned(const void *p, int64_t ld) { return !p || (host::aligned16(p) && ld % 8 == 0); }

}  // namespace

bool linear_layout_fits(const LinearParams &p) {
    return rows_aligned(p.x, p.ldx) && rows_aligned(p.w, p.ldw) && rows_aligned(p.out, p.ldo) &&
           rows_aligned(p.preact, p.ldp) && rows_aligned(p.aux, p.ldaux);
}

bool linear_prefers_split(const LinearParams &p, int num_sms) {
    (void)num_sms;
    // the tiles' outputs leave by tensor copies, which write whole 16-byte units: a row
    // that ends inside one would have up to 7 elements past its end overwritten
    if (p.n % 8 != 0) return true;
    return p.m <= 256;
}

cudaError_t launch_linear_split(bool bf16, const LinearParams &lp, int num_sms, cudaStream_t stream) {
    const SplitShape s = split_shape(lp, num_sms);
    if (s.tiles * s.split > INT32_MAX) return cudaErrorInvalidValue;
    SplitParams p = {};
    const uint64_t m = lp.m, n = lp.n, k = lp.k;
    bool ok = host::make_map16(&p.x_map, lp.x, k, m, kDepth, static_cast<uint32_t>(s.rows), lp.ldx);
    ok = ok && (lp.w_nk ? host::make_map16(&p.w_map, lp.w, k, n, kDepth, kTileN, lp.ldw)
                        : host::make_map16(&p.w_map, lp.w, n, k, 64, kDepth, lp.ldw));
    if (!ok) return cudaErrorInvalidValue;
    p.bias = lp.bias, p.aux = lp.aux_mode == AUX_NONE ? nullptr : lp.aux, p.out = lp.out, p.preact = lp.preact;
    p.ldaux = lp.ldaux, p.ldo = lp.ldo, p.ldp = lp.ldp;
    p.m = lp.m, p.n = lp.n;
    p.steps = (lp.k + kDepth - 1) / kDepth;
    p.w_kn = !lp.w_nk;
    p.rows = s.rows, p.m_tiles = s.m_tiles, p.split = s.split;
    p.stages = s.stages, p.accs = s.accs, p.tmem_cols = s.tmem_cols;
    p.aligned = 1;   // linear_layout_fits
    p.act = activation_of(lp.act);
    p.status = device_status_word();
    p.wait_limit_ns = host::kWaitLimitNs;
    if (lp.aux_mode == AUX_ACT_GRAD)
        return bf16 ? launch_split<true, EPI_BACKWARD>(p, s, stream) : launch_split<false, EPI_BACKWARD>(p, s, stream);
    return bf16 ? launch_split<true, EPI_FORWARD>(p, s, stream) : launch_split<false, EPI_FORWARD>(p, s, stream);
}

}  // namespace mc2
