"""The Python calls around the linears on the GPU: the regular case (marshalled
by the extension module) and the others (by the Python code) give the same
results, and refusals come with their own errors from both."""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

B = torch.bfloat16


def tensors(m=12, h=256, n=136):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(m, h, generator=g).to(B).cuda()
    return x, torch.ones(h, dtype=B, device="cuda"), (torch.randn(n, h, generator=g) * h ** -0.5).to(B).cuda()


def slices(x):
    """x as a (3, 4, h) tensor of strided rows: rows of one stride, but not a matrix."""
    wide = torch.zeros(3, 4, x.shape[1] + 8, dtype=x.dtype, device=x.device)
    wide[:, :, :x.shape[1]] = x.view(3, 4, -1)
    return wide[:, :, :x.shape[1]]


def test_rows_of_one_stride_in_more_dimensions():
    x, w, lin = tensors()
    s = slices(x)
    a = mc2.mc2_add_rms_norm(x, w, residual=x, with_rstd=True, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, with_out=1)
    b = mc2.mc2_add_rms_norm(s, w, residual=s, with_rstd=True, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, with_out=1)
    for name in ("out", "residual", "rstd", "q", "scale"):
        assert torch.equal(a[name].reshape(-1), b[name].reshape(-1)), name
    ga, wa = mc2.mc2_rms_norm_grad(x, a["residual"], w, a["rstd"], dres=x)
    gb, wb = mc2.mc2_rms_norm_grad(s, b["residual"], w, b["rstd"], dres=s)
    assert torch.equal(ga.view(-1), gb.reshape(-1)) and torch.equal(wa, wb)
    oa, pa = mc2.mc2_matmul_bias_act(x, lin, activation="silu", with_preact=True)
    ob, pb = mc2.mc2_matmul_bias_act(s, lin, activation="silu", with_preact=True)
    assert torch.equal(oa.view(-1), ob.view(-1)) and torch.equal(pa.view(-1), pb.view(-1))
    za = mc2.mc2_matmul_act_grad(oa, lin, x, activation="gelu")
    zb = mc2.mc2_matmul_act_grad(ob, lin, s, activation="gelu")
    assert torch.equal(za.view(-1), zb.view(-1))
    assert torch.equal(mc2.mc2_act_grad(x, x, activation="relu").view(-1), mc2.mc2_act_grad(s, s, activation="relu").view(-1))


def test_given_outputs_are_used_and_returned():
    x, w, lin = tensors()
    out, ro, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(12, device="cuda")
    q, sc = torch.empty(12, 256, dtype=torch.int8, device="cuda"), torch.empty(12, 2, device="cuda")
    r = mc2.mc2_add_rms_norm(x, w, residual=x, quant_mode=mc2.QUANT_PERGROUP, out=out, residual_out=ro, rstd=rstd, q=q, scale=sc)
    assert r["out"] is out and r["residual"] is ro and r["rstd"] is rstd and r["q"] is q and r["scale"] is sc
    f = mc2.mc2_add_rms_norm(x, w, residual=x, quant_mode=mc2.QUANT_PERGROUP, with_out=True, with_rstd=True)
    for name in r:
        assert torch.equal(r[name], f[name]), name
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(mc2.mc2_rms_norm_grad_workspace(12, 256), dtype=torch.uint8, device="cuda")
    a = mc2.mc2_rms_norm_grad(x, x, w, rstd, dx=dx, dw=dw, workspace=ws)
    b = mc2.mc2_rms_norm_grad(x, x, w, rstd)
    assert a[0] is dx and a[1] is dw and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, p = torch.empty(12, 136, dtype=B, device="cuda"), torch.empty(12, 136, dtype=B, device="cuda")
    a = mc2.mc2_matmul_bias_act(x, lin, activation="gelu", out=o, preact=p)
    b = mc2.mc2_matmul_bias_act(x, lin, activation="gelu", with_preact=True)
    assert a[0] is o and a[1] is p and torch.equal(o, b[0]) and torch.equal(p, b[1])


def test_refusals():
    x, w, lin = tensors()
    cpu = x.cpu()
    for f, match in ((lambda: mc2.mc2_add_rms_norm(cpu, w), "x must be a CUDA tensor"),
                     (lambda: mc2.mc2_add_rms_norm(x, w[:255]), "weight must have shape"),
                     (lambda: mc2.mc2_add_rms_norm(x, w, residual=x.float()), "residual must be of dtype"),
                     (lambda: mc2.mc2_add_rms_norm(x.t(), w[:12]), "rows of adjacent elements"),
                     (lambda: mc2.mc2_add_rms_norm(x, w, q=x), "need a quant_mode"),
                     (lambda: mc2.mc2_rms_norm_grad(x, x, w, torch.zeros(12, dtype=B, device="cuda")), "rstd must be of dtype"),
                     (lambda: mc2.mc2_matmul_bias_act(x, lin.t()), "w must have shape"),
                     (lambda: mc2.mc2_matmul_bias_act(x, lin, bias=w), "bias must have shape"),
                     (lambda: mc2.mc2_matmul_bias_act(x, lin, activation="tanh"), "activation must be one of"),
                     (lambda: mc2.mc2_matmul_act_grad(x, lin, x, activation="relu"), "w must have shape"),
                     (lambda: mc2.mc2_act_grad(x, x[:5], activation="relu"), "z must have shape")):
        with pytest.raises(ValueError, match=match):
            f()
    for f, status in ((lambda: mc2.mc2_add_rms_norm(x, w, eps=-1.0), mc2.MC2_ERR_SHAPE),
                      (lambda: mc2.mc2_add_rms_norm(x, w, quant_mode=mc2.QUANT_MX, q_dtype=torch.int8), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_add_rms_norm(x, w, quant_mode=3), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_add_rms_norm(x[:0], w), mc2.MC2_ERR_SHAPE),
                      (lambda: mc2.mc2_add_rms_norm(x, w.half()), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_rms_norm_grad(x, x, w, torch.ones(12, device="cuda"), workspace=w), mc2.MC2_ERR_WORKSPACE),
                      (lambda: mc2.mc2_matmul_bias_act(x.float(), lin.float()), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_matmul_bias_act(x[:0], lin), mc2.MC2_ERR_SHAPE),
                      (lambda: mc2.mc2_act_grad(x[:0], x[:0], activation="silu"), mc2.MC2_ERR_SHAPE)):
        with pytest.raises(mc2.Mc2Error) as e:
            f()
        assert e.value.status == status and e.value.message


def test_calls_in_a_cuda_graph():
    """Captured and replayed on new inputs: the calls neither synchronise nor allocate outside the capture's pool."""
    x, w, lin = tensors(m=5)
    down = (lin.t().contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            n = mc2.mc2_add_rms_norm(x, w, residual=x)
            h, _ = mc2.mc2_matmul_bias_act(n["out"], lin, activation="silu")
            mc2.mc2_matmul_bias_act(h, down, residual=n["residual"])
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n = mc2.mc2_add_rms_norm(x, w, residual=x)
        h, _ = mc2.mc2_matmul_bias_act(n["out"], lin, activation="silu")
        y, _ = mc2.mc2_matmul_bias_act(h, down, residual=n["residual"])
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        n2 = mc2.mc2_add_rms_norm(x, w, residual=x)
        h2, _ = mc2.mc2_matmul_bias_act(n2["out"], lin, activation="silu")
        y2, _ = mc2.mc2_matmul_bias_act(h2, down, residual=n2["residual"])
        assert torch.equal(y, y2)
