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
// Which of the two is expected to be faster for these sizes.
bool linear_prefers_split(const LinearParams &p, int num_sms);

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
