// linear.h -- the fused-epilogue matrix product's kernels, as the C entry points call them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mc2 {

// What the epilogue does with the second matrix it reads (aux, the shape of out):
//   AUX_NONE      out = act(acc + bias)
//   AUX_RESIDUAL  out = act(acc + bias) + aux
//   AUX_ACT_GRAD  out = acc * act'(aux)
enum AuxMode : int { AUX_NONE = 0, AUX_RESIDUAL = 1, AUX_ACT_GRAD = 2 };

// out (m, n) from x (m, k) and w, (n, k) when w_nk or (k, n); strides are in
// elements, from row to row.  All tensors are of one 16-bit type.
struct LinearParams {
    const void *x, *w, *bias, *aux;
    void *out, *preact;
    int64_t ldx, ldw, ldaux, ldo, ldp;
    int m, n, k;
    int w_nk;
    int act;        // ActKind
    int aux_mode;   // AuxMode
    // a product of int8 codes: out, aux and a 16-bit bias of the given type, z = float(acc) x_scale w_scale + bias.  The split
    // kernel takes x and w as they are (16-byte aligned, strides a multiple of 16; out and aux of any layout), the tiles as fp16
    int codes;
    const float *x_scale, *w_scale;   // (m), (n)
    int bias_f32;
};

// Any sizes and layouts, without tensor cores.
cudaError_t launch_linear_any(bool bf16, const LinearParams &p, cudaStream_t stream);

// The tensor-core kernels take 16-byte aligned matrices whose strides are multiples
// of 8 elements and below 2^39 (the tensor copies' rule), and sizes that leave a tile
// of room in 32 bits; the strides of single rows are set by the caller.
bool linear_layout_fits(const LinearParams &p);
// Depth of one accumulator of the 256 x 256 tiles, in 64-deep stages: the contraction in blocks of 2048, whose sums are
// added in fp32 with round-to-nearest.  The tensor core cuts each sum it adds to 24 bits, which
// takes 5.8e-6 of a sum of one sign for each 1024 deep, always towards zero; an epilogue (5 to 8 us)
// hides behind the next tile's first block (9 us).  A rest of at most half a block is spread
// over the others: a short last block leaves the tensor cores waiting for the one before to be read (8192 x 8192
// x 2112 170 us, 155 as one block).
inline int linear_tiles_block(int k) {
    const int steps = (k + 63) / 64, blocks = (steps + 15) / 32;
    const int even = blocks > 1 ? (steps + blocks - 1) / blocks : steps;
    return even > 32 || blocks <= 1 ? even : 32;
}
// A CTA pair per 256 x 256 tile: products of many rows.
cudaError_t launch_linear_tiles(bool bf16, const LinearParams &p, cudaStream_t stream);
// The weight's columns as the tile's rows, the contraction split over a cluster:
// products whose tiles would not fill the device.
cudaError_t launch_linear_split(bool bf16, const LinearParams &p, int num_sms, cudaStream_t stream);
// What the split kernel is expected to take for codes, in us; negative where it cannot sum them exactly.
float linear_split_codes_us(const LinearParams &p);
// Which of the two is expected to be faster for these sizes.
bool linear_prefers_split(const LinearParams &p, int num_sms);

// The sums of dy^T x, (n, k), over parts of the m rows, each to a matrix of its own in `parts` (fp32, rows ldp apart), and
// dy's column sums, in weight_grad_col_parts shares a part, to col_parts (splits x shares, n) if given.  A part is split_blocks blocks of block_tiles 64-row stages; a
// block's sum stays in one accumulator, blocks are added in fp32 to nearest.
struct WeightGradParts {
    const void *dy, *x;
    float *parts, *col_parts;
    int64_t lddy, ldx, ldp;
    int m, n, k;
    int splits, split_blocks, block_tiles;
};
cudaError_t launch_weight_grad_parts(bool bf16, const WeightGradParts &w, cudaStream_t stream);
inline int weight_grad_col_parts(int k) { return (k + 255) / 256; }
// The whole of it in 16 bits: dw (n, k) with rows of a multiple of 8 elements, dw 16-byte aligned; db (n) or none, or its
// shares in col_parts (weight_grad_col_parts, n) instead.
cudaError_t launch_weight_grad_tiles(bool bf16, const void *dy, int64_t lddy, const void *x, int64_t ldx, int m, int n, int k, void *dw,
                                     void *db, float *col_parts, int num_sms, cudaStream_t stream);

// dz = dy * act'(z), (m, n)
struct ActGradParams {
    const void *dy, *z;
    void *dz;
    int64_t lddy, ldz, lddz;
    int64_t m, n;
    int act;
};
cudaError_t launch_act_grad(bool bf16, const ActGradParams &p, int num_sms, cudaStream_t stream);

}  // namespace mc2
