// quant_linear.cu -- products of 8-bit codes: the int8 product with scales per token and per channel, and the weight
// gradient whose input is kept in 8 bits.
//
//   out[t, j] = act(float(sum_l x[t, l] W[l, j]) x_scale[t] w_scale[j] + bias[j]) + residual[t, j]
//   dw[i, j]  = sum_t dy[t, i] act(q[t, j] scale),  db[i] = sum_t dy[t, i]
//
// The tensor cores take 16-bit operands (their int8 rate is a tenth of it here).  int8 codes are exact in fp16, and so are
// the fp32 sums of 1024 of their products; act(q scale) is rounded to dy's type.  The codes of few tokens are widened on
// their way to the tensor cores (linear_split.cu): the weight is read once, as bytes.  The operands of many rows are
// brought to 16 bits in the workspace, each element once, and multiplied by the GEMM of gemm_tcgen05.cuh; matrices that the
// tensor copies cannot take go through the workspace, too.  4096 tokens, 7168 x 8192: 282 to 295 us, of which widening takes 43; the
// weight gradient 4096 x 7168 of 8192 tokens 286 us, from gelu(z) 294 to 303 (its values 36 and 44 us), the product itself 250.
#include "kept.h"

#include "codes.cuh"
#include "host.h"
#include "linear.h"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kThreads = 256;
constexpr int kSms = 152, kPairs = kSms / 2;   // of a GB300 (the plans, and so the workspace queries, ask no device: here or in linear_split.cu)

// A matrix of int8 and where it goes, in rows `pitch` apart (a multiple of 16): as fp16, or as it is.
struct Widened {
    const int8_t *src;
    void *dst;
    int64_t ld, pitch, rows;
    int64_t cols;
    int64_t vectors;   // of a row: 8 columns each as fp16, 16 as they are (16 bytes written)
    int whole;         // one row of whole vectors, 16-byte aligned
};

// Both operands of a product in one launch: blocks [0, first) take a, the others b, 16 bytes written a thread at a time, so that
// a warp's stores are one stretch (92 M codes: 55 us with two of them a thread, 32 bytes apart, 43 this way, 6.4 TB/s).
template <bool kWiden>
__global__ void __launch_bounds__(kThreads) widen_kernel(const __grid_constant__ Widened a, const __grid_constant__ Widened b, int first) {
    constexpr int kVector = kWiden ? 8 : 16, kAhead = 4;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const bool is_a = static_cast<int>(blockIdx.x) < first;
    const Widened &t = is_a ? a : b;
    const int64_t block = is_a ? blockIdx.x : blockIdx.x - first, blocks = is_a ? first : gridDim.x - first;
    const int64_t total = t.rows * t.vectors, step = blocks * kThreads;
    int64_t e = block * kThreads + threadIdx.x;
    if (kWiden && t.whole) {
        uint4 *to = static_cast<uint4 *>(t.dst);
        const uint2 *from = reinterpret_cast<const uint2 *>(t.src);
        for (; e + (kAhead - 1) * step < total; e += kAhead * step) {
            uint2 q[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) q[i] = from[e + i * step];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const uint2 lo = widen4(q[i].x), hi = widen4(q[i].y);
                to[e + i * step] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
    for (; e < total; e += step) {
        int64_t r = 0, v = e;
        if (t.rows > 1) {
            if (total <= UINT32_MAX) {
                r = static_cast<uint32_t>(e) / static_cast<uint32_t>(t.vectors);
            } else {
                r = e / t.vectors;
            }
            v = e - r * t.vectors;
        }
        // (a row's last vector is whole, zeros behind its end)
        const int64_t left = t.cols - v * kVector;
        const uint4 q = load_codes16(t.src + r * t.ld + v * kVector, left < kVector ? static_cast<int>(left) : kVector);
        if constexpr (kWiden) {
            const uint2 lo = widen4(q.x), hi = widen4(q.y);
            *reinterpret_cast<uint4 *>(static_cast<__half *>(t.dst) + r * t.pitch + v * kVector) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<int8_t *>(t.dst) + r * t.pitch + v * kVector) = q;
        }
    }
}

// Rows of 16-bit elements from one layout to another, by the aligned 16-byte units of the destination's rows (the first and
// the last of them partial): a warp a row at a time.
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const uint16_t *src, int64_t lds, uint16_t *dst, int64_t ldd, int64_t rows, int cols) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = kThreads / 32;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * warps + warp; r < rows; r += static_cast<int64_t>(gridDim.x) * warps) {
        const uint16_t *from = src + r * lds;
        uint16_t *to = dst + r * ldd;
        for (int j = lane * 8 - static_cast<int>((reinterpret_cast<uintptr_t>(to) >> 1) & 7); j < cols; j += 32 * 8) {
            if (j >= 0 && j + 8 <= cols) {
                *reinterpret_cast<uint4 *>(to + j) = load_codes16(reinterpret_cast<const int8_t *>(from + j), 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j + e >= 0 && j + e < cols) to[j + e] = from[j + e];
            }
        }
    }
}

// dw and db from the parts' sums, added in order (db's are col_count).  Four columns a thread; rows of dw are k elements, of a
// part ldp.
template <bool kBF16>
__global__ void __launch_bounds__(kThreads) add_parts_kernel(const float *parts, int64_t ldp, int splits, int n, int k, void *dw,
                                                             const float *col_parts, int col_count, void *db, int dw_blocks) {
    using T = typename Elem<kBF16 ? ELEM_BF16 : ELEM_F16>::type;
    using E = Elem<kBF16 ? ELEM_BF16 : ELEM_F16>;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    if (static_cast<int>(blockIdx.x) >= dw_blocks) {
        // 32 columns a block, a warp every eighth share, then the warps' sums in order
        __shared__ float sums[kThreads / 32][32];
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = (blockIdx.x - dw_blocks) * 32 + lane;
        float s = 0.0f;
        if (i < n) {
#pragma unroll 4
            for (int p = warp; p < col_count; p += kThreads / 32) s = __fadd_rn(s, col_parts[static_cast<int64_t>(p) * n + i]);
        }
        sums[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && i < n) {
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) s = __fadd_rn(s, sums[w][lane]);
            E::store(static_cast<T *>(db) + i, s);
        }
        return;
    }
    const int64_t quads = (k + 3) / 4, total = quads * n, part = ldp * n;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < total; e += static_cast<int64_t>(dw_blocks) * kThreads) {
        const int64_t r = e / quads;
        const int c = static_cast<int>(e - r * quads) * 4;
        const float4 *from = reinterpret_cast<const float4 *>(parts + r * ldp + c);
        float4 s = *from;
#pragma unroll 4
        for (int p = 1; p < splits; ++p) {
            const float4 t = from[p * (part / 4)];
            s.x = __fadd_rn(s.x, t.x), s.y = __fadd_rn(s.y, t.y), s.z = __fadd_rn(s.z, t.z), s.w = __fadd_rn(s.w, t.w);
        }
        T *to = static_cast<T *>(dw) + r * k + c;
        const float v[4] = {s.x, s.y, s.z, s.w};
        if (c + 4 <= k && (reinterpret_cast<uintptr_t>(to) & 7u) == 0) {
            T o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) E::store(&o[i], v[i]);
            *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(o);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < k) E::store(to + i, v[i]);
        }
    }
}

template <class... A>
cudaError_t launch(void (*kern)(A...), int64_t grid, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

int64_t blocks_for(int64_t items, int num_sms) {
    const int64_t blocks = (items + kThreads - 1) / kThreads, most = 32ll * num_sms;
    return blocks < 1 ? 1 : (blocks < most ? blocks : most);
}

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// What the tensor copies take: 16-byte aligned, rows a multiple of 16 bytes (and less than 2^40) apart; writes go in units of
// 16 bytes, so an output's rows are whole units.
bool copies_read16(const void *p, int64_t ld, int64_t rows) {
    return host::aligned16(p) && (rows == 1 || (ld % 8 == 0 && ld < (1ll << 39)));
}
bool copies_read8(const void *p, int64_t ld, int64_t rows) {
    return host::aligned16(p) && (rows == 1 || (ld % 16 == 0 && ld < (1ll << 40)));
}
bool copies_write16(const void *p, int64_t ld, int64_t rows, int64_t cols) { return copies_read16(p, ld, rows) && cols % 8 == 0; }

// Pieces of a workspace, 256-byte aligned to one another.
struct Pieces {
    size_t total = 0;
    size_t take(int64_t elems, size_t size) {
        const size_t at = total;
        total += (static_cast<size_t>(elems) * size + 255) / 256 * 256;
        return at;
    }
};

// The matrices and sizes as the product kernels take them.
LinearParams product_of(const QuantProduct &p) {
    LinearParams l = {};
    l.m = p.m, l.n = p.n, l.k = p.k;
    l.w_nk = p.w_nk;
    l.act = p.act;
    l.bias = p.bias, l.bias_f32 = p.bias_f32;
    l.aux_mode = p.residual ? AUX_RESIDUAL : AUX_NONE;
    l.codes = 1, l.x_scale = p.x_scale, l.w_scale = p.w_scale;
    return l;
}

// A contraction over m rows for few outputs is split: parts of it on CTA pairs that would have no tile, and their sums added by
// a kernel of their own.  In us: 6.3 and 0.29 a 64-row stage for each wave of tiles (as in linear_prefers_split), and for the parts their
// bytes, written and read, at 5000 a ns, and a launch.
struct WeightPlan {
    size_t x = 0, dy = 0, parts = 0, col_parts = 0, total = 0;
    bool dy_apart = false, in_parts = false;
    int col_count = 0;   // shares of db (0: it is written as it is)
    int splits = 1, split_blocks = 1, block_tiles = 16;
};

WeightPlan plan_weight_grad(const QuantWeightGrad &p) {
    WeightPlan at;
    const int64_t tiles = ((p.n + 255ll) / 256) * ((p.k + 255ll) / 256);
    const int steps = (p.m + 63) / 64;
    const bool whole = copies_write16(p.dw, p.k, p.n, p.k);
    float best = 0.0f;
    for (int s = 1; s <= 32 && s <= steps; ++s) {
        const float waves = static_cast<float>((tiles * s + kPairs - 1) / kPairs);
        float us = 6.3f + 0.29f * waves * static_cast<float>((steps + s - 1) / s);
        if (s > 1 || !whole) us += 3.0f + static_cast<float>(s) * static_cast<float>(p.n) * static_cast<float>(p.k) * 8.0f / 5.0e6f;
        if (s == 1 || us < best) best = us, at.splits = s;
    }
    at.in_parts = at.splits > 1 || !whole;
    if (at.in_parts) {
        // equal blocks of at most 2048 rows (as the tiles of linear.h's products), a whole number of them a part
        const int each = (steps + at.splits - 1) / at.splits;
        at.split_blocks = (each + 31) / 32;
        at.block_tiles = (each + at.split_blocks - 1) / at.split_blocks;
        const int blocks = (steps + at.block_tiles - 1) / at.block_tiles;
        at.splits = (blocks + at.split_blocks - 1) / at.split_blocks;
    }
    Pieces ws;
    at.x = ws.take(p.m * up8(p.k), 2);
    at.dy_apart = !copies_read16(p.dy, p.lddy, p.m);
    if (at.dy_apart) at.dy = ws.take(p.m * up8(p.n), 2);
    if (at.in_parts) at.parts = ws.take(static_cast<int64_t>(at.splits) * p.n * ((p.k + 3ll) / 4 * 4), 4);
    // db in shares of the columns of tiles: at no cost where the parts are added anyway, for a launch (2 us) otherwise, which
    // pays from 1024 rows on (8192 x 1024 x 4096 73 -> 59 us, 1024 x 4096 x 4096 34.4 and 34)
    const int shares = weight_grad_col_parts(p.k);
    if (at.in_parts || (steps >= 16 && shares > 1)) {
        at.col_count = at.splits * shares;
        at.col_parts = ws.take(static_cast<int64_t>(at.col_count) * p.n, 4);
    }
    at.total = ws.total;
    return at;
}

}  // namespace

ProductPlan plan_quant_product(const QuantProduct &p) {
    ProductPlan at;
    // one to four tokens (4096 x 4096: 4.3, 4.6 and 7.9 us for 1, 2 and 4, 7.9 in the kernel of few; 28672 x 8192 42.9, 43.9 and 55, there
    // 49.5, but here a weight of any alignment is read as it is); to eight where the weight is small (1024 x 8192 5.5 against 6.7)
    at.tokens = p.w_nk && (p.m <= 4 || (p.m <= 8 && static_cast<int64_t>(p.n) * p.k <= 8ll << 20));
    if (at.tokens) return at;
    // Which kernel, by the sizes alone: the tiles take 9.4 us, 3.2 and 0.25 a 64-deep stage for each wave of them, and widening three
    // bytes a code at 6400 a ns (1024 tokens, 8192 x 4096 65 us; 2048 and 4096 tokens, 4096 x 4096 59.5 and 102).  Where the two
    // cross, with k = 4096: 512 tokens, n = 4096 30.5 us split, 37 in tiles; 1024 tokens, n = 8192 65 in tiles.
    const int64_t tiles = ((p.m + 255ll) / 256) * ((p.n + 255ll) / 256);
    const float steps = static_cast<float>((p.k + 63) / 64);
    const float tiles_us = 9.4f + static_cast<float>((tiles + kPairs - 1) / kPairs) * (3.2f + 0.2475f * steps) +
                           (static_cast<float>(p.m) + static_cast<float>(p.n)) * static_cast<float>(p.k) * 0.47e-6f;
    const float split_us = linear_split_codes_us(product_of(p));
    at.split = split_us >= 0.0f && split_us < tiles_us;
    Pieces ws;
    const int64_t w_rows = p.w_nk ? p.n : p.k, w_cols = p.w_nk ? p.k : p.n;
    at.x_apart = !at.split || !copies_read8(p.x, p.ldx, p.m);
    at.w_apart = !at.split || !copies_read8(p.w, p.ldw, w_rows);
    if (at.x_apart) at.x = ws.take(p.m * up16(p.k), at.split ? 1 : 2);
    if (at.w_apart) at.w = ws.take(w_rows * up16(w_cols), at.split ? 1 : 2);
    if (!at.split) {
        at.out_apart = !copies_write16(p.out, p.ldo, p.m, p.n);
        at.residual_in = p.residual && (at.out_apart || !copies_read16(p.residual, p.ldr, p.m));
        if (at.out_apart) at.out = ws.take(p.m * up8(p.n), 2);
    }
    at.total = ws.total;
    return at;
}

cudaError_t launch_quant_product(bool bf16, const QuantProduct &p, const ProductPlan &at, int num_sms, cudaStream_t stream, Mark mark, void *ctx) {
    if (at.tokens) {
        const cudaError_t e = launch_quant_tokens(bf16, p, stream);
        if (e == cudaSuccess) mark(ctx);
        return e;
    }
    char *ws = static_cast<char *>(p.workspace);
    LinearParams l = product_of(p);
    const int64_t w_rows = p.w_nk ? p.n : p.k, w_cols = p.w_nk ? p.k : p.n;
    cudaError_t e = cudaSuccess;
    // (the stride of a single row is free: one that the tensor copies take)
    l.x = p.x, l.ldx = p.m == 1 ? up16(p.k) : p.ldx;
    l.w = p.w, l.ldw = w_rows == 1 ? up16(w_cols) : p.ldw;
    if (at.x_apart || at.w_apart) {
        const auto taken = [&](const int8_t *src, int64_t ld, void *dst, int64_t rows, int64_t cols) {
            const int vector = at.split ? 16 : 8;
            Widened t = {src, dst, ld, up16(cols), rows, cols, (cols + vector - 1) / vector, 0};
            // matrices without gaps are one row
            if (ld == cols && cols % 16 == 0) {
                t.cols = rows * cols, t.rows = 1, t.vectors = t.cols / vector;
                t.whole = host::aligned16(src);
            }
            return t;
        };
        const Widened a = taken(p.x, p.ldx, ws + at.x, p.m, p.k), b = taken(p.w, p.ldw, ws + at.w, w_rows, w_cols);
        // blocks in proportion to the elements, at least one for each operand that is taken
        const int64_t na = at.x_apart ? a.rows * a.vectors : 0, nb = at.w_apart ? b.rows * b.vectors : 0, blocks = blocks_for(na + nb, num_sms) + 1;
        int64_t first = static_cast<int64_t>(static_cast<double>(blocks) * na / (na + nb) + 0.5);
        const int64_t least = na ? 1 : 0, most = nb ? blocks - 1 : blocks;
        first = first < least ? least : (first > most ? most : first);
        e = launch(at.split ? widen_kernel<false> : widen_kernel<true>, blocks, stream, a, b, static_cast<int>(first));
        if (e != cudaSuccess) return e;
        mark(ctx);
        if (at.x_apart) l.x = ws + at.x, l.ldx = up16(p.k);
        if (at.w_apart) l.w = ws + at.w, l.ldw = up16(w_cols);
    }
    if (at.split) {
        l.out = p.out, l.ldo = p.ldo, l.aux = p.residual, l.ldaux = p.ldr;
        e = launch_linear_split(bf16, l, kSms, stream);
        if (e == cudaSuccess) mark(ctx);
        return e;
    }
    void *out = at.out_apart ? static_cast<void *>(ws + at.out) : p.out;
    const int64_t ldo = at.out_apart || p.m == 1 ? up8(p.n) : p.ldo;
    if (at.residual_in) {
        e = launch(copy_rows_kernel, blocks_for(static_cast<int64_t>(p.m) * 32, num_sms), stream, static_cast<const uint16_t *>(p.residual), p.ldr,
                   static_cast<uint16_t *>(out), ldo, static_cast<int64_t>(p.m), p.n);
        if (e != cudaSuccess) return e;
        mark(ctx);
    }
    l.out = out, l.ldo = ldo;
    l.aux = at.residual_in ? out : p.residual;
    l.ldaux = at.residual_in ? ldo : (p.m == 1 ? up8(p.n) : p.ldr);
    e = launch_linear_tiles(bf16, l, stream);
    if (e != cudaSuccess) return e;
    mark(ctx);
    if (at.out_apart) {
        e = launch(copy_rows_kernel, blocks_for(static_cast<int64_t>(p.m) * 32, num_sms), stream, static_cast<const uint16_t *>(out), ldo, static_cast<uint16_t *>(p.out),
                   p.ldo, static_cast<int64_t>(p.m), p.n);
        if (e != cudaSuccess) return e;
        mark(ctx);
    }
    return cudaSuccess;
}

size_t quant_weight_grad_workspace(const QuantWeightGrad &p) { return plan_weight_grad(p).total; }

cudaError_t launch_quant_weight_grad(bool bf16, const QuantWeightGrad &p, int num_sms, cudaStream_t stream, Mark mark, void *ctx) {
    const WeightPlan at = plan_weight_grad(p);
    char *ws = static_cast<char *>(p.workspace);
    // act(q scale) is rounded to dy's type, the tensor cores' operand type, as an activation kept in 16 bits would be.  With the output's
    // own rounding dw is then 2.3e-3 off (bf16; 2.9e-4 fp16; 2-norm, relative), 1.7e-3 (2.1e-4) without it; the eight bits
    // that q was kept in cost more.  A second operand for the bits that are dropped would double the product, 250 us of 296.
    const int64_t ldx = up8(p.k);
    cudaError_t e = launch_act_dequant(bf16 ? ELEM_BF16 : ELEM_F16, p.x, p.act, ws + at.x, ldx, num_sms, stream);
    if (e != cudaSuccess) return e;
    mark(ctx);
    const void *dy = p.dy;
    int64_t lddy = p.m == 1 ? up8(p.n) : p.lddy;
    if (at.dy_apart) {
        dy = ws + at.dy, lddy = up8(p.n);
        e = launch(copy_rows_kernel, blocks_for(static_cast<int64_t>(p.m) * 32, num_sms), stream, static_cast<const uint16_t *>(p.dy), p.lddy,
                   reinterpret_cast<uint16_t *>(ws + at.dy), lddy, static_cast<int64_t>(p.m), p.n);
        if (e != cudaSuccess) return e;
        mark(ctx);
    }
    float *col_parts = p.db && at.col_count ? reinterpret_cast<float *>(ws + at.col_parts) : nullptr;
    const float *parts = nullptr;
    const int64_t ldp = (p.k + 3ll) / 4 * 4;
    if (at.in_parts) {
        WeightGradParts w = {};
        w.dy = dy, w.x = ws + at.x, w.parts = reinterpret_cast<float *>(ws + at.parts), w.col_parts = col_parts;
        w.lddy = lddy, w.ldx = ldx, w.ldp = ldp;
        w.m = p.m, w.n = p.n, w.k = p.k;
        w.splits = at.splits, w.split_blocks = at.split_blocks, w.block_tiles = at.block_tiles;
        parts = w.parts;
        e = launch_weight_grad_parts(bf16, w, stream);
    } else {
        e = launch_weight_grad_tiles(bf16, dy, lddy, ws + at.x, ldx, p.m, p.n, p.k, p.dw, p.db, col_parts, num_sms, stream);
    }
    if (e != cudaSuccess) return e;
    mark(ctx);
    if (!parts && !col_parts) return cudaSuccess;
    const int64_t dw_blocks = parts ? blocks_for(p.n * ((p.k + 3ll) / 4), num_sms) : 0, db_blocks = col_parts ? (p.n + 31) / 32 : 0;
    e = launch(bf16 ? add_parts_kernel<true> : add_parts_kernel<false>, dw_blocks + db_blocks, stream, parts, ldp, at.splits, p.n, p.k, p.dw,
               static_cast<const float *>(col_parts), at.col_count, p.db, static_cast<int>(dw_blocks));
    if (e == cudaSuccess) mark(ctx);
    return e;
}

}  // namespace mc2
