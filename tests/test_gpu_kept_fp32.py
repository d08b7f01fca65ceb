"""mc2_act_dequant with an output of 32 bits: activations to fp32's precision, relative to the value, far below zero too.

Bounds, relative to act of the fp32 z.  gelu: CUDA's normcdff is within 5 steps (2^-23 each), one product 2^-24.  silu: expf within
2 steps, in the numerator and (at most half of it) in the denominator, three more roundings of 2^-24: 4.5 2^-23.  gelu_tanh: that, and
e^-|v|'s error from v's, whose constants and products are six roundings: 6 |v| 2^-24.  Subnormal values and factors: a few of
2^-149 times |z| <= 104: 2^-140.
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu


def plain(z, act):
    if act == "gelu":
        return z * torch.special.erfc(-z * 0.5 ** 0.5) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("h", [256, 250])   # whole chunks, and any layout
def test_precision_relative_to_the_value(act, h):
    q = torch.arange(-127, 128, dtype=torch.int8).repeat(2)[:h].repeat(64, 1).contiguous().cuda()
    scale = torch.logspace(-4, 0, 64).float().cuda()   # to -127
    out = mc2.mc2_act_dequant(q, scale, activation=act, dtype=torch.float32)
    z = (q.float() * scale[:, None]).double()
    ref = plain(z, act)
    v = 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3).abs().clamp(max=110)
    relative = {"gelu": 5.5 * 2.0 ** -23, "silu": 4.5 * 2.0 ** -23, "gelu_tanh": 4.5 * 2.0 ** -23 + 6 * v.clamp(max=110) * 2.0 ** -24}[act]
    bad = ~((out.double() - ref).abs() <= relative * ref.abs() + 2.0 ** -140)
    assert not bad.any(), (int(bad.sum()), z[bad][:4].tolist(), out[bad][:4].tolist(), ref[bad][:4].tolist())


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("h", [256, 250])
def test_the_ends(act, h):
    """Infinities give their limits, a NaN stays in its element, large values are themselves."""
    q = torch.ones(6, h, dtype=torch.int8, device="cuda")
    q[:, 1] = -1
    scale = torch.tensor([float("inf"), float("nan"), 3.0e38, 1e20, 1e-45, 200.0], device="cuda")
    out = mc2.mc2_act_dequant(q, scale, activation=act, dtype=torch.float32)
    assert (out[0, 2:] == float("inf")).all() and out[0, 1] == 0 and out[1].isnan().all()
    for row in (2, 3, 5):
        assert (out[row, 2:] == scale[row]).all() and out[row, 1] == 0
    assert (out[4].abs() <= scale[4]).all()
