"""mc2_matmul_weight_grad_quant gives the same bits in every call, beside another stream's work too, and its outputs are off by the
roundings that its comment names: that of act(q scale) to the operands' type and that of the output.

The error of rounding a value x of [1, 2) is spread evenly over [-UNIT, UNIT], so its relative mean square is UNIT^2 / (3 x^2), on
average over the binade UNIT^2 / 6.  Two independent roundings, the first of each term of a sum of terms of either sign: sqrt(2 / 6) UNIT =
0.58 UNIT in the 2-norm; 0.65 leaves room for the fp32 sums and the values' distribution.
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
TOKEN, GROUP, MX = mc2.QUANT_PERTOKEN_DYNAMIC, mc2.QUANT_PERGROUP, mc2.QUANT_MX


@pytest.mark.parametrize("m,n,k,dtype,act,mode", [(8192, 4096, 7168, BF16, "gelu", GROUP), (333, 1000, 4104, F16, "none", TOKEN),
                                                  (16384, 512, 1024, BF16, "none", MX), (3000, 1001, 257, BF16, "silu", TOKEN)])
def test_the_same_bits_each_time(m, n, k, dtype, act, mode):
    g = torch.Generator(device="cuda").manual_seed(m)
    q, scale = mc2.mc2_act_quant(torch.randn(m, k, generator=g, device="cuda"), quant_mode=mode,
                                 q_dtype=torch.float8_e4m3fn if mode == MX else torch.int8)
    dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(dtype)
    dw, db = mc2.mc2_matmul_weight_grad_quant(dy, q, scale, activation=act)
    side, big = torch.cuda.Stream(), torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(20):
        with torch.cuda.stream(side):
            big[: 1 << 26].copy_(big[1 << 26:])
        w, b = mc2.mc2_matmul_weight_grad_quant(dy, q, scale, activation=act)
        bad += (w.view(torch.int16) != dw.view(torch.int16)).sum() + (b.view(torch.int16) != db.view(torch.int16)).sum()
    assert int(bad) == 0
    steps = scale.double() if mode != MX else torch.ldexp(torch.ones_like(scale, dtype=torch.float64), scale.int() - 127)
    z = q.double() * steps.view(m, -1).repeat_interleave({TOKEN: k, GROUP: 128, MX: 32}[mode], 1)[:, :k]
    a = z if act == "none" else z * torch.sigmoid(z) if act == "silu" else z * torch.special.erfc(-z * 0.5 ** 0.5) / 2
    ref = dy.double().t() @ a
    off = float((dw.double() - ref).norm() / ref.norm())
    assert off <= 0.65 * (2.0 ** -8 if dtype == BF16 else 2.0 ** -11), off
