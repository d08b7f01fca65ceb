"""Calls with ``stream=``: their workspace and new outputs belong to that stream, so
what the current stream allocates meanwhile is other memory."""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

B = torch.bfloat16
BUSY = 200_000_000   # clocks: a tenth of a second


def behind(stream):
    """A stream with work on it that the next call waits for."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)


def fill(sizes, value=7):
    """Tensors of these sizes on the current stream, filled now."""
    return [torch.full((n,), value, dtype=torch.uint8, device="cuda") for n in sizes]


def untouched(tensors, value=7):
    return all(bool((t == value).all()) for t in tensors)


@pytest.mark.parametrize("w_is_strided", [False, True])
def test_gradient_workspace_on_a_side_stream(w_is_strided):
    """Both marshalling paths: a matrix, and rows of one stride in three dimensions."""
    m, h = 1000, 2048
    g = torch.Generator().manual_seed(0)
    x, dy, dres = ((torch.randn(m, h, generator=g)).to(B).cuda() for _ in range(3))
    w = torch.ones(h, dtype=B, device="cuda")
    rstd = mc2.mc2_add_rms_norm(x, w, with_rstd=True)["rstd"]
    dx, dw = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres)
    size = mc2.mc2_rms_norm_grad_workspace(m, h)
    if w_is_strided:
        wide = torch.zeros(10, 100, h + 8, dtype=B, device="cuda")
        wide[:, :, :h] = x.view(10, 100, h)
        x, dy, dres, rstd = wide[:, :, :h], dy.view(10, 100, h), dres.view(10, 100, h), rstd.view(10, 100)
    fill([size, size])   # (freed again: blocks of this size that an allocation here would take)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    behind(s)
    gx, gw = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres, stream=s)
    mine = fill([size] * 4)
    torch.cuda.synchronize()
    assert untouched(mine)
    assert torch.equal(gw, dw) and torch.equal(gx.reshape(m, h), dx)


@pytest.mark.parametrize("mode", [mc2.QUANT_PERTOKEN_DYNAMIC, mc2.QUANT_PERTOKEN])
def test_all_to_all_workspace_on_a_side_stream(mode):
    ranks, m, h, n = 4, 256, 256, 512
    g = torch.Generator().manual_seed(1)
    dtype = B if mode == mc2.QUANT_PERTOKEN_DYNAMIC else torch.int8
    chunks = [(torch.randn(m, h, generator=g) * (1 if dtype == B else 40)).clamp(-127, 127).to(dtype).cuda() for _ in range(ranks)]
    x2 = torch.randint(-127, 128, (ranks * h, n), generator=g, dtype=torch.int8).cuda()
    s2, bias = torch.rand(n, generator=g).cuda() * 1e-3, torch.randn(n, generator=g).cuda()
    kw = dict(x1_quant_mode=mode)
    if mode == mc2.QUANT_PERTOKEN:
        kw["x1_scale"] = torch.rand(m, generator=g).cuda()
    want = mc2.mc2_alltoall_quant_mm(chunks, x2, s2, bias, **kw)["out"]
    size = mc2.mc2_alltoall_quant_mm_workspace(ranks, m, h, n, mode, dtype)
    fill([size, size])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    behind(s)
    got = mc2.mc2_alltoall_quant_mm(chunks, x2, s2, bias, stream=s, **kw)["out"]
    mine = fill([size] * 4)
    torch.cuda.synchronize()
    assert untouched(mine) and torch.equal(got, want)


def calls():
    """Each call that makes outputs: f(stream) and its outputs as a list."""
    g = torch.Generator().manual_seed(2)

    def t(*shape, std=1.0, dtype=B):
        return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

    x, w1, lin, z = t(512, 256), torch.ones(256, dtype=B, device="cuda"), t(256, 256, std=1 / 16), t(512, 256)
    rstd = mc2.mc2_add_rms_norm(x, w1, with_rstd=True)["rstd"]
    codes = [torch.randint(-127, 128, (64, 1024), generator=g, dtype=torch.int8).cuda() for _ in range(2)]
    scales = [torch.rand(64, 8, generator=g).cuda() for _ in range(2)]
    return {
        "add_rms_norm": lambda s: mc2.mc2_add_rms_norm(x, w1, residual=z, with_rstd=True, quant_mode=mc2.QUANT_PERGROUP,
                                                       with_out=True, stream=s).values(),
        "rms_norm_grad": lambda s: mc2.mc2_rms_norm_grad(z, x, w1, rstd, stream=s),
        "matmul_bias_act": lambda s: mc2.mc2_matmul_bias_act(x, lin, activation="silu", with_preact=True, stream=s),
        "matmul_act_grad": lambda s: [mc2.mc2_matmul_act_grad(x, lin, z, activation="silu", stream=s)],
        "act_grad": lambda s: [mc2.mc2_act_grad(x, z, activation="gelu", stream=s)],
        "all_gather_mm": lambda s: mc2.mc2_all_gather_mm([x, z], lin, stream=s),
        "matmul_reduce_scatter": lambda s: mc2.mc2_matmul_reduce_scatter([x, z], [lin, lin], stream=s),
        "matmul_weight_grad": lambda s: mc2.mc2_matmul_weight_grad(x, z, stream=s),
        "quant_all_reduce": lambda s: [mc2.mc2_quant_all_reduce(codes, scales, stream=s)],
    }


@pytest.mark.parametrize("name", ["add_rms_norm", "rms_norm_grad", "matmul_bias_act", "matmul_act_grad", "act_grad",
                                  "all_gather_mm", "matmul_reduce_scatter", "matmul_weight_grad", "quant_all_reduce"])
def test_outputs_on_a_side_stream(name):
    """A new output is no block that the current stream still writes, and stays while that
    stream, which has waited, still reads it."""
    f = calls()[name]
    want = [t.clone() for t in f(None)]
    sizes = [t.nbytes for t in want]
    s, home = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    # blocks of these sizes, freed while the current stream has still to write them
    torch.cuda._sleep(BUSY)
    fill(sizes)
    got = list(f(s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # read behind work here and freed before that is done: what s allocates then is other memory
    del got
    got = list(f(s))
    home.wait_stream(s)
    torch.cuda._sleep(BUSY)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        fill([n for n in sizes for _ in range(4)], 5)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))


def test_a_given_output_and_the_current_stream_itself():
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(3)).to(B).cuda()
    w = torch.ones(256, dtype=B, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(x)
    want = mc2.mc2_add_rms_norm(x, w)["out"]
    torch.cuda.synchronize()
    assert mc2.mc2_add_rms_norm(x, w, out=out, stream=s)["out"] is out
    s.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(mc2.mc2_add_rms_norm(x, w, stream=torch.cuda.current_stream())["out"], want)
