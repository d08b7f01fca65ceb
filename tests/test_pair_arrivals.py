"""Pairs of CTAs that widen int8 codes: what one CTA's warps write, the other CTA's warp has multiplied, so what tells it
publishes to the cluster."""
import glob
import os
import re

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

CSRC = os.path.join(os.path.dirname(os.path.abspath(mc2.__file__)), "csrc")


def test_no_arrival_at_another_cta_publishes_to_its_own_only():
    for f in glob.glob(os.path.join(CSRC, "*.cu*")):
        assert not re.search(r"arrive\.(release\.cta|release|noComplete)?\.?shared::cluster", open(f).read()), os.path.basename(f)


@pytest.mark.gpu
@pytest.mark.parametrize("w_is_nk", [True, False])
@pytest.mark.parametrize("m,n,k", [(65, 2048, 4096), (96, 4096, 1024), (130, 1024, 8192), (256, 4096, 4096), (300, 2560, 2048),
                                   (512, 4096, 2048)])
def test_many_products_under_load(m, n, k, w_is_nk):
    """Exact sums in every one of many products, of codes that change from one to the next, beside another stream's copies
    and products."""
    g = torch.Generator().manual_seed(m)
    codes = [torch.randint(-127, 128, (m, k), generator=g, dtype=torch.int8).cuda() for _ in range(6)]
    weights = [torch.randint(-127, 128, (n, k) if w_is_nk else (k, n), generator=g, dtype=torch.int8).cuda() for _ in range(4)]
    one, scale = torch.full((m,), 2.0 ** -14, device="cuda"), torch.ones(n, device="cuda")
    want = [[((x.double() @ (w.double().t() if w_is_nk else w.double())) * 2.0 ** -14).to(torch.bfloat16) for w in weights] for x in codes]
    side, big = torch.cuda.Stream(), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(240):
        if i % 4 == 0:
            with torch.cuda.stream(side):
                big[: 1 << 27].copy_(big[1 << 27:])
                mc2.mc2_quant_matmul(codes[0], one, weights[0], scale, w_is_nk=w_is_nk)
        x, w = i % 6, i % 4
        bad += (mc2.mc2_quant_matmul(codes[x], one, weights[w], scale, w_is_nk=w_is_nk) != want[x][w]).sum()
    torch.cuda.synchronize()
    assert int(bad) == 0 and mc2.mc2_device_status() == mc2.MC2_OK
