"""How deep a product of many rows sums in one accumulator of the tensor core.

Bounds.  As in the other tests of these products a sum of d terms on the tensor
core (16 terms a step) is within (d/16 + 16) 2^-23 of the sum of its terms'
sizes, of which cutting towards zero takes its share at every step.  Here d is
one block of the contraction (2048, and half as much again where a rest is
spread); the n blocks are added in fp32 to nearest, n 2^-24.

The terms have one sign, so nothing averages out, and the residual takes the nearest fp16
value of the product off again: the output holds what is left, to 2^-11 of itself.
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BLOCK = 2048


def terms_of_one_sign(m, n, k, w_is_nk):
    g = torch.Generator().manual_seed(k)
    x = (torch.rand(m, k, generator=g) * 0.5 + 0.5).half().cuda()
    w = ((torch.rand(n, k, generator=g) * 0.5 + 0.5) * (64 / k)).half().cuda()
    return x, w if w_is_nk else w.t().contiguous(), x.double() @ w.double().t()


# outputs of more than one wave of 256 x 256 tiles: one block, several, and rests that are spread
@pytest.mark.parametrize("m,n,k", [(2048, 2560, 2048), (2048, 2560, 2560), (2048, 2560, 7168), (2300, 2304, 8200),
                                   (2560, 2048, 24576)])
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_sums_are_no_deeper_than_a_block(m, n, k, w_is_nk):
    x, w, z = terms_of_one_sign(m, n, k, w_is_nk)
    near = z.half()
    left = z - near.double()
    depth, blocks = min(k, BLOCK * 3 // 2), -(-k // BLOCK)
    sums = ((depth / 16 + 16) * 2.0 ** -23 + (blocks + 1) * 2.0 ** -24) * z   # (and one for the residual)
    out, _ = mc2.mc2_matmul_bias_act(x, w, w_is_nk=w_is_nk, residual=-near)
    off = (out.double() - left).abs()
    bound = sums * (1 + 2.0 ** -11) + 2.0 ** -11 * left.abs() + 2.0 ** -25
    assert bool((off <= bound).all()), f"{float((off / bound).max()):.3g} of the bound, {float((off / z).max()):.3g} of the sum"
    # the gradient's product of the same sums
    got = mc2.mc2_matmul_act_grad(x, w, torch.ones_like(near), activation="relu", w_is_nk=not w_is_nk)
    assert bool(((got.double() - z).abs() <= sums + 2.0 ** -11 * (z + sums)).all())
