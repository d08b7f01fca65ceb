"""The norm's codes where the other calls take them: per-token int8 into
AlltoAllQuantMatmul's full-quant mode, per-group and mx codes into
QuantAllReduce; and the example that runs everything."""
import os
import subprocess
import sys

import pytest
import torch

import oracle
import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_codes_into_the_full_quant_product():
    """Bit for bit the oracle's product of the same codes and scales."""
    g = torch.Generator().manual_seed(0)
    m, ranks, h, n = 130, 4, 128, 256
    x = torch.randn(m, ranks * h, generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(ranks * h, dtype=torch.bfloat16, device="cuda")
    c = mc2.mc2_add_rms_norm(x, w, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC)
    chunks = [c["q"][:, r * h:(r + 1) * h].contiguous() for r in range(ranks)]
    x2 = torch.randint(-127, 128, (ranks * h, n), generator=g, dtype=torch.int8)
    s2, bias = torch.rand(n, generator=g) * 1e-3, torch.randn(n, generator=g)
    out = mc2.mc2_alltoall_quant_mm(chunks, x2.cuda(), s2.cuda(), bias.cuda(), x1_quant_mode=mc2.QUANT_PERTOKEN,
                                    x1_scale=c["scale"])["out"]
    ref = oracle.alltoall_quant_mm([k.cpu() for k in chunks], x2, s2, bias, quant_mode=3, x1_scale=c["scale"].cpu())
    assert torch.equal(out.cpu().view(torch.int16), ref["out"].view(torch.int16))


@pytest.mark.parametrize("mode,q_dtype", [(mc2.QUANT_PERGROUP, torch.int8), (mc2.QUANT_PERGROUP, torch.float8_e5m2),
                                          (mc2.QUANT_MX, torch.float8_e4m3fn)])
def test_codes_into_the_quantised_all_reduce(mode, q_dtype):
    """The sum of two ranks' codes is the sum of their outputs, to the codes' own error: half
    a step of 1/127 of the group's largest value (int8), half of 2^-2 (e5m2), half of 2^-3
    with saturation at 1.75 / 2 of the top binade (mx e4m3), each relative, on each rank."""
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(9, 1024, generator=g).cuda() for _ in range(2)]
    w = torch.ones(1024, device="cuda")
    rs = [mc2.mc2_add_rms_norm(x, w, quant_mode=mode, q_dtype=q_dtype, with_out=True) for x in xs]
    scales = [r["scale"].view(9, 16, 2) if mode == mc2.QUANT_MX else r["scale"] for r in rs]
    out = mc2.mc2_quant_all_reduce([r["q"] for r in rs], scales, out_dtype=torch.float32)
    bound = torch.zeros(9, 1024, device="cuda", dtype=torch.float64)
    for r in rs:
        v = r["out"].double()
        if q_dtype == torch.int8:
            bound += v.view(9, 8, 128).abs().amax(2).repeat_interleave(128, 1) / 254
        else:
            top = v.view(9, -1, 128 if mode == mc2.QUANT_PERGROUP else 32).abs().amax(2)
            top = top.repeat_interleave(1024 // top.shape[1], 1)
            bound += v.abs() / (8 if q_dtype == torch.float8_e5m2 else 16) + top * 2.0 ** -16
            if mode == mc2.QUANT_MX:
                bound += (v.abs() - 0.875 * 2 * torch.exp2(torch.floor(torch.log2(top)))).clamp(min=0)
    want = rs[0]["out"].double() + rs[1]["out"].double()
    assert ((out.double() - want).abs() <= bound * (1 + 1e-5) + 1e-6).all()


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "mlp_block.py"), "--tokens", "200", "--hidden", "1024", "--ffn", "2048"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "one token, captured" in r.stdout
