"""mc2_rms_norm_grad where each block takes many rows: the ring's stages are used
again, its shares of dw grow over the rows, and rows are read ahead of stores that may
go to their tensor.  The bounds are those of test_gpu_rms_norm.py."""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2
from test_gpu_rms_norm import BF16, E, F16, F32, LEAST, UNIT, make, near, plain_grad

pytestmark = pytest.mark.gpu

# at most 152 blocks of 1024 threads, 304 of 512, ..., 1216 of 128 and fewer (one vector a thread): 4 to 13 rows a block
ALIGNED = [(9000, 256), (5000, 136), (6100, 1024), (2000, 4096), (1200, 8192), (700, 12288), (620, 16384)]
# rows that are no whole vectors: 4, 8 and 16 columns a thread, and beyond
ODD = [(7000, 77), (6000, 1003), (900, 5003), (700, 8195), (500, 20000), (610, 16387)]


def check(m, h, dtype, w_f32, with_dres, over=None, wide=0):
    x, dres, w = make(m, h, dtype, seed=m + h, residual=with_dres, w_f32=w_f32, wide=wide)
    dy, _, _ = make(m, h, dtype, seed=m + h + 1, residual=False, wide=wide)
    rstd = mc2.mc2_add_rms_norm(x, w, with_rstd=True)["rstd"]
    rdx, size, rdw, wsize = plain_grad(dy, x, w, rstd, dres)
    target = {None: None, "dy": dy, "x": x, "dres": dres}[over]
    dx, dw = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres, dx=target)
    if target is not None:
        assert dx is target
        if wide:
            assert bool((target._base[:, h:] == 7).all())
    near(dx, rdx, UNIT[dtype], "dx", E(h) * size + LEAST[dtype])
    near(dw, rdw, UNIT[w.dtype], "dw", (m + 310) * 2.0 ** -24 * wsize + LEAST[w.dtype])


@pytest.mark.parametrize("m,h", ALIGNED + ODD)
@pytest.mark.parametrize("dtype,w_f32", [(BF16, False), (F16, True), (F32, True)])
@pytest.mark.parametrize("with_dres", [False, True])
def test_many_rows_a_block(m, h, dtype, w_f32, with_dres):
    check(m, h, dtype, w_f32, with_dres)


@pytest.mark.parametrize("m,h", [(9000, 256), (2000, 4096), (700, 12288), (6000, 1003), (700, 8195), (500, 20000)])
@pytest.mark.parametrize("over", ["dy", "x", "dres"])
def test_in_place_over_many_rows(m, h, over):
    check(m, h, BF16, False, True, over=over)


@pytest.mark.parametrize("m,h", [(2000, 4096), (6000, 1003)])
@pytest.mark.parametrize("over", ["x", "dres"])
def test_in_place_in_strided_rows(m, h, over):
    check(m, h, F16, False, True, over=over, wide=8)


@pytest.mark.parametrize("m,h", [(1, 4096), (5, 1000), (21, 1003), (3, 20000)])
@pytest.mark.parametrize("over", ["x", "dres"])
def test_in_place_over_few_rows(m, h, over):
    check(m, h, BF16, False, True, over=over)


@pytest.mark.parametrize("m,h", [(2000, 4096), (6000, 1003)])
def test_same_bits_every_time(m, h):
    x, dres, w = make(m, h, BF16, seed=1)
    dy, _, _ = make(m, h, BF16, seed=2, residual=False)
    rstd = mc2.mc2_add_rms_norm(x, w, with_rstd=True)["rstd"]
    a = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres)
    b = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
