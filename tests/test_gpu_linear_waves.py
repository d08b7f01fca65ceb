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
