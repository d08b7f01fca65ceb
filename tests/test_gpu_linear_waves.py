"""Products whose 256 x 256 tiles come in several waves: each CTA pair takes tile
after tile, so what its epilogue carries from one to the next counts.  The values
are small integers: every sum is exact in fp32 and every output in 16 bits, so
the outputs are compared bit for bit.
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def integers(m, n, k, dtype, w_is_nk, seed=0):
    """The sums' deviation is below 35, so that they stay within what bf16 holds exactly."""
    g = torch.Generator().manual_seed(seed + m + n + k)
    x = torch.randint(-2, 3, (m, k), generator=g).to(dtype).cuda()
    w = (torch.randint(-2, 3, (n, k), generator=g) * (torch.rand(n, k, generator=g) < min(0.1, 300 / k))).to(dtype)
    w = (w if w_is_nk else w.t().contiguous()).cuda()
    bias = torch.randint(-3, 4, (n,), generator=g).to(dtype).cuda()
    res = torch.randint(-4, 5, (m, n), generator=g).to(dtype).cuda()
    z = x.float() @ (w.float().t() if w_is_nk else w.float()) + bias.float()   # exact: integers below 2^24
    assert float(z.abs().max()) <= 240
    return x, w, bias, res, z


# last column tiles of 1, 2, 3 and 4 pieces of 32 columns, in the first half and the second
WIDTHS = [5128, 5168, 5192, 5240, 5256, 5336, 5376]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("use_res,use_pre", [(False, False), (False, True)])
def test_last_column_tiles(n, use_res, use_pre):
    m, k = 5000, 72
    x, w, bias, res, z = integers(m, n, k, BF16, True)
    for _ in range(3):
        out, pre = mc2.mc2_matmul_bias_act(x, w, bias=bias, activation="relu", residual=res if use_res else None,
                                           with_preact=use_pre)
        assert torch.equal(out.float(), z.clamp(min=0) + (res.float() if use_res else 0))
        if use_pre:
            assert torch.equal(pre.float(), z)


@pytest.mark.parametrize("m,n,k", [(5000, 5000, 136), (4100, 6152, 264)])
@pytest.mark.parametrize("w_is_nk", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("use_res,use_pre,in_place", [(False, False, False), (False, True, False), (True, False, False),
                                                      (True, True, False), (True, False, True), (True, True, True)])
def test_forms_over_several_waves(m, n, k, w_is_nk, dtype, use_res, use_pre, in_place):
    """Ragged last row and column tiles, in each form of the epilogue."""
    x, w, bias, res, z = integers(m, n, k, dtype, w_is_nk)
    want = z.clamp(min=0) + (res.float() if use_res else 0)
    out, pre = mc2.mc2_matmul_bias_act(x, w, w_is_nk=w_is_nk, bias=bias, activation="relu", residual=res if use_res else None,
                                       with_preact=use_pre, out=res if in_place else None)
    assert torch.equal(out.float(), want)
    if use_pre:
        assert torch.equal(pre.float(), z)


@pytest.mark.parametrize("k", [2048, 2056, 2112, 3136, 4096, 4200, 6208, 8200])
@pytest.mark.parametrize("use_res,use_pre", [(False, True), (True, False)])
def test_blocks_of_the_contraction(k, use_res, use_pre):
    """One to four blocks, whose last may be shorter, over two or three tiles a CTA pair."""
    x, w, bias, res, z = integers(5000, 2088, k, BF16, True)
    out, pre = mc2.mc2_matmul_bias_act(x, w, bias=bias, activation="relu", residual=res if use_res else None, with_preact=use_pre)
    assert torch.equal(out.float(), z.clamp(min=0) + (res.float() if use_res else 0))
    if use_pre:
        assert torch.equal(pre.float(), z)
    y = torch.ones_like(res)
    assert torch.equal(mc2.mc2_matmul_act_grad(x, w, y, activation="relu", w_is_nk=False).float(), z - bias.float())


@pytest.mark.parametrize("m,n,k", [(300, 520, 20000), (64, 264, 72000), (1, 136, 70000), (512, 2048, 12296), (128, 1032, 33000)])
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_accumulators_used_again(m, n, k, w_is_nk):
    """Few rows, and contractions of more 1024-deep parts than the few-row kernel has accumulators."""
    x, w, bias, res, z = integers(m, n, k, BF16, w_is_nk)
    out, pre = mc2.mc2_matmul_bias_act(x, w, w_is_nk=w_is_nk, bias=bias, activation="relu", residual=res, with_preact=True)
    assert torch.equal(out.float(), z.clamp(min=0) + res.float()) and torch.equal(pre.float(), z)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("use_res,use_pre", [(False, False), (True, True)])
def test_activations_over_several_waves(act, use_res, use_pre):
    """The same bits as in 16 calls of few rows each, whose epilogue is the other kernel's: the sums are exact in both."""
    m, n, k = 5000, 5000, 136
    x, w, bias, res, z = integers(m, n, k, F16, True)
    out, pre = mc2.mc2_matmul_bias_act(x, w, bias=bias, activation=act, residual=res if use_res else None, with_preact=use_pre)
    for r in range(0, m, 313):
        part, _ = mc2.mc2_matmul_bias_act(x[r:r + 313], w, bias=bias, activation=act, residual=res[r:r + 313] if use_res else None)
        assert torch.equal(out[r:r + 313], part)
    if use_pre:
        assert torch.equal(pre.float(), z)
