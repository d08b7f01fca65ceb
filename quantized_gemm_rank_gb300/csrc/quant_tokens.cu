// quant_tokens.cu -- the int8 product of one to eight tokens with an (n, k) weight.
//
//   out[t, j] = act(float(sum_l x[t, l] w[j, l]) x_scale[t] w_scale[j] + bias[j]) + residual[t, j]
//
// Reading the weight once bounds it, so there is nothing between memory and the sums: a lane takes 16 codes of each of
// four rows of the weight at a time, and the same 16 of every token (from L1), and adds their products four at a time
// (dp4a, exact int32).  One token, 4096 x 4096: 4.3 us, 28672 x 4096 22.6 (5.2 TB/s), 28672 x 8192 42 to 43 (5.5), weights by turns that L2 does
// not hold.  The tensor cores need the codes widened and an accumulator's way back: 7.9 us for 4096 x 4096 in linear_split.cu.  Rows share a block by slices of the depth, joined through shared memory.
#include "kept.h"

#include "codes.cuh"
#include "host.h"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;      // of the weight, a warp
constexpr int kTurn = 512;    // codes of a row that a warp takes at a time
// Turns on their way at once, and blocks an SM holds: bytes in flight, which need registers, against warps, which do, too (one
// token, 4096 x 4096: 3.7 us with four blocks, 6.4 with three).
__host__ __device__ constexpr int turns_ahead(int tokens) { return tokens <= 2 ? 2 : 1; }
constexpr int resident(int tokens) { return tokens <= 2 ? 4 : (tokens <= 4 ? 3 : 2); }

// kAligned: every row begins at a multiple of 16 bytes.
template <bool kBF16, int kM, bool kAligned>
__global__ void __launch_bounds__(kThreads, resident(kM)) quant_tokens_kernel(const __grid_constant__ QuantProduct p, Activation act, int slices,
                                                                              int slice) {
    using E = Elem<kBF16 ? ELEM_BF16 : ELEM_F16>;
    using T = typename E::type;
    constexpr int kAhead = turns_ahead(kM), kBatch = kM < 4 ? kM : 4;
    __shared__ int parts[kWarps][kRows * kM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / slices, s = warp - group * slices, groups = kWarps / slices;
    const int j0 = (blockIdx.x * groups + group) * kRows;
    const int k0 = s * slice + lane * 16, k1 = min(p.k, (s + 1) * slice);
    const int8_t *w = p.w + j0 * p.ldw + k0;
    if (lane % 8 == 0 && k0 < k1) {
        // the first turn's lines into L2 while the stream's previous kernel ends (nothing is read by this)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (j0 + r < p.n) ptx::prefetch_l2(w + r * p.ldw);
    }
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    int acc[kRows][kM] = {};
    const int8_t *x = p.x + k0;
    const auto load = [](const int8_t *from, int left, bool again) {
        if (kAligned && left >= 16) return again ? *reinterpret_cast<const uint4 *>(from) : load_once(from);
        return load_codes16(from, left, again);
    };
    for (int k = k0; k < k1; k += kAhead * kTurn) {
        uint4 q[kAhead][kRows];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
            for (int r = 0; r < kRows; ++r) q[a][r] = load(w + r * p.ldw + a * kTurn, j0 + r < p.n ? k1 - k - a * kTurn : 0, false);
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
            for (int b = 0; b < kM; b += kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int t = 0; t < kBatch; ++t) v[t] = load(x + (b + t) * p.ldx + a * kTurn, b + t < p.m ? k1 - k - a * kTurn : 0, true);
#pragma unroll
                for (int t = 0; t < kBatch; ++t)
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        int &sum = acc[r][b + t];
                        sum = __dp4a(static_cast<int>(q[a][r].x), static_cast<int>(v[t].x), sum);
                        sum = __dp4a(static_cast<int>(q[a][r].y), static_cast<int>(v[t].y), sum);
                        sum = __dp4a(static_cast<int>(q[a][r].z), static_cast<int>(v[t].z), sum);
                        sum = __dp4a(static_cast<int>(q[a][r].w), static_cast<int>(v[t].w), sum);
                    }
            }
        w += kAhead * kTurn, x += kAhead * kTurn;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int t = 0; t < kM; ++t) {
            const int sum = __reduce_add_sync(0xFFFFFFFFu, acc[r][t]);
            if (lane == 0) parts[warp][t * kRows + r] = sum;
        }
    __syncthreads();
    // two outputs a thread, of neighbouring rows of the weight: an activation works on pairs, and these are the pairs of the
    // other kernels (a last column without a neighbour has a zero beside it)
    static_assert(kRows % 2 == 0, "pairs within a warp's rows");
    for (int e = threadIdx.x; e < groups * (kRows / 2) * kM; e += kThreads) {
        const int t = e / (groups * (kRows / 2)), g = (e / (kRows / 2)) % groups, r = e % (kRows / 2) * 2;
        const int j = (blockIdx.x * groups + g) * kRows + r;
        if (t >= p.m || j >= p.n) continue;
        float z[2] = {};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (j + c >= p.n) continue;
            int sum = 0;
            for (int i = 0; i < slices; ++i) sum += parts[g * slices + i][t * kRows + r + c];
            z[c] = __fmul_rn(__fmul_rn(__int2float_rn(sum), p.x_scale[t]), p.w_scale[j + c]);
            if (p.bias)
                z[c] = __fadd_rn(z[c], p.bias_f32 ? static_cast<const float *>(p.bias)[j + c] : E::load(static_cast<const T *>(p.bias) + j + c));
        }
        const float2 a = act2(make_float2(z[0], z[1]), act);
        const float o[2] = {a.x, a.y};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (j + c >= p.n) continue;
            float v = o[c];
            if (p.residual) v = __fadd_rn(v, E::load(static_cast<const T *>(p.residual) + t * p.ldr + j + c));
            E::store(static_cast<T *>(p.out) + t * p.ldo + j + c, v);
        }
    }
}

template <bool kBF16, int kM, bool kAligned>
cudaError_t launch_tokens(const QuantProduct &p, cudaStream_t stream) {
    // slices of the depth of at least two turns, a power of two of them a block
    int slices = 1;
    while (slices < kWarps && p.k > slices * 2 * kTurn) slices *= 2;
    const int turns = (p.k + kTurn - 1) / kTurn, slice = (turns + slices - 1) / slices * kTurn;
    const int rows = kWarps / slices * kRows;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((p.n + rows - 1) / rows), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, quant_tokens_kernel<kBF16, kM, kAligned>, p, activation_of(p.act), slices, slice);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kBF16, int kM>
cudaError_t launch_tokens(const QuantProduct &p, cudaStream_t stream) {
    const auto whole = [](const void *q, int64_t ld, int rows) { return host::aligned16(q) && (rows == 1 || ld % 16 == 0); };
    return whole(p.x, p.ldx, p.m) && whole(p.w, p.ldw, p.n) ? launch_tokens<kBF16, kM, true>(p, stream) : launch_tokens<kBF16, kM, false>(p, stream);
}

}  // namespace

cudaError_t launch_quant_tokens(bool bf16, const QuantProduct &p, cudaStream_t stream) {
    if (p.m == 1) return bf16 ? launch_tokens<true, 1>(p, stream) : launch_tokens<false, 1>(p, stream);
    if (p.m == 2) return bf16 ? launch_tokens<true, 2>(p, stream) : launch_tokens<false, 2>(p, stream);
    if (p.m <= 4) return bf16 ? launch_tokens<true, 4>(p, stream) : launch_tokens<false, 4>(p, stream);
    return bf16 ? launch_tokens<true, 8>(p, stream) : launch_tokens<false, 8>(p, stream);
}

}  // namespace mc2
