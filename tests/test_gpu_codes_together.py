"""The calls on 8-bit codes as a block uses them: an MLP served in int8 from the norm to the residual, and its training step
whose activations are kept in 8 bits; captured in a graph, on other streams, several at once, and through both of the binding's
marshalling paths.  Each call is compared, from the codes that it was given, with a plain one in 64 bits (bounds as in
the calls' own tests: one rounding of the output, and of a weight gradient's operand)."""
import threading

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

B = torch.bfloat16
TOKEN, GROUP, MX = mc2.QUANT_PERTOKEN_DYNAMIC, mc2.QUANT_PERGROUP, mc2.QUANT_MX


def gelu(z):
    return z * torch.special.erfc(-z * 0.5 ** 0.5) / 2


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def values(q, scale):
    k = q.shape[-1]
    s = scale.double()
    if scale.dtype == torch.uint8:
        s = torch.ldexp(torch.ones_like(s), scale.int() - 127).repeat_interleave(32, -1)[..., :k]
    elif scale.dim() == q.dim():
        s = s.repeat_interleave(128, -1)[..., :k]
    else:
        s = s[..., None]
    return q.double() * s


class Mlp:
    def __init__(self, hidden, ffn, seed=0):
        g = torch.Generator().manual_seed(seed)

        def t(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(B).cuda()

        self.norm, self.b1 = 1 + t(hidden, std=0.1), t(ffn, std=0.1)
        self.w1, self.w2 = t(ffn, hidden, std=hidden ** -0.5), t(hidden, ffn, std=ffn ** -0.5)
        self.q1, self.s1 = mc2.mc2_act_quant(self.w1)   # a weight's rows are its channels
        self.q2, self.s2 = mc2.mc2_act_quant(self.w2)

    def serve(self, x, **kw):
        n = mc2.mc2_add_rms_norm(x, self.norm, residual=x, quant_mode=TOKEN, **kw)
        z = mc2.mc2_quant_matmul(n["q"], n["scale"], self.q1, self.s1, bias=self.b1, **kw)
        q, s = mc2.mc2_act_quant(z, activation="gelu", **kw)
        y = mc2.mc2_quant_matmul(q, s, self.q2, self.s2, residual=n["residual"], **kw)
        return n, z, q, s, y

    def step(self, x, dy, mode, kind):
        """Forward in int8, the pre-activation kept; backward from what was kept."""
        n, z, _, _, y = self.serve(x)
        kept = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind)
        dw2, db2 = mc2.mc2_matmul_weight_grad_quant(dy, *kept, activation="gelu")
        dh, _ = mc2.mc2_matmul_bias_act(dy, self.w2, w_is_nk=False)
        dz = mc2.mc2_act_grad_quant(dh.clone(), *kept, activation="gelu")
        dw1, db1 = mc2.mc2_matmul_weight_grad_quant(dz, n["q"], n["scale"])
        return dict(n=n, z=z, kept=kept, dh=dh, dz=dz, dw1=dw1, db1=db1, dw2=dw2, db2=db2, y=y)


@pytest.mark.parametrize("m", [1, 3, 7, 40, 300, 2500])
def test_an_mlp_served_in_int8(m):
    b = Mlp(512, 1536)
    x = torch.randn(m, 512, generator=torch.Generator().manual_seed(m)).to(B).cuda()
    n, z, q, s, y = b.serve(x)
    z64 = values(n["q"], n["scale"]) @ values(b.q1, b.s1).t() + b.b1.double()
    y64 = values(q, s) @ values(b.q2, b.s2).t() + n["residual"].double()
    assert off(z, z64) < 2.0 ** -8 and off(y, y64) < 2.0 ** -8
    # the codes are those of gelu(z): half a step of a row's largest value, and z's own error
    h = gelu(z.double())
    top = h.abs().amax(1, keepdim=True)
    assert ((values(q, s) - h).abs() <= top / 254 * (1 + 2.0 ** -12) + 2.0 ** -18 * (1 + z.double().abs())).all()
    # int8 codes of rows of 512 normal values: each rounded to 1/127 of the row's largest, about 3.2 of them: 1% of a row's norm
    # through each of four operands
    full = gelu(n["residual"].double() / torch.sqrt(n["residual"].double().square().mean(1, keepdim=True) + 1e-6) * b.norm.double() @ b.w1.double().t()
                + b.b1.double()) @ b.w2.double().t()
    assert off(y.double() - n["residual"].double(), full) < 0.05


@pytest.mark.parametrize("mode,kind", [(TOKEN, torch.int8), (GROUP, torch.int8), (GROUP, torch.float8_e4m3fn), (MX, torch.float8_e4m3fn)])
@pytest.mark.parametrize("m", [5, 333])
def test_a_training_step_from_kept_codes(m, mode, kind):
    b = Mlp(264, 1000)
    g = torch.Generator().manual_seed(m)
    x, dy = torch.randn(m, 264, generator=g).to(B).cuda(), (torch.randn(m, 264, generator=g) * 0.1).to(B).cuda()
    r = b.step(x, dy, mode, kind)
    z = values(*r["kept"]).requires_grad_()
    gelu(z).sum().backward()
    assert off(r["dz"], r["dh"].double() * z.grad) < 2.0 ** -8
    assert off(r["dw2"], dy.double().t() @ gelu(z.detach())) < 1.5 * 2.0 ** -8
    assert off(r["dw1"], r["dz"].double().t() @ values(r["n"]["q"], r["n"]["scale"])) < 1.5 * 2.0 ** -8
    assert off(r["db2"], dy.double().sum(0)) < 2.0 ** -8 and off(r["db1"], r["dz"].double().sum(0)) < 2.0 ** -8


@pytest.mark.parametrize("m", [1, 6, 48, 700])
def test_captured_and_replayed(m):
    """On new inputs, twice; the graph's own memory holds the workspaces."""
    b = Mlp(512, 1024)
    g = torch.Generator().manual_seed(3)
    x, dy = torch.randn(m, 512, generator=g).to(B).cuda(), torch.randn(m, 512, generator=g).to(B).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(x, dy, GROUP, torch.int8)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):   # two graphs of the same call, alive at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = b.step(x, dy, GROUP, torch.int8)
        graphs.append((graph, r))
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        for graph, _ in graphs:
            graph.replay()
        want = b.step(x, dy, GROUP, torch.int8)
        for _, r in graphs:
            for name in ("y", "z", "dz", "dw1", "db1", "dw2", "db2"):
                assert torch.equal(r[name], want[name]), name


def test_on_several_streams_and_threads_at_once():
    """Products whose CTAs share SMs and tensor memory, from threads of their own: the bits of a call by itself."""
    b = Mlp(1024, 2048)
    xs = [torch.randn(m, 1024, generator=torch.Generator().manual_seed(m)).to(B).cuda() for m in (16, 64, 130, 260, 900, 3)]
    want = [b.serve(x)[4] for x in xs]
    grads = [mc2.mc2_matmul_weight_grad_quant(x, *mc2.mc2_act_quant(x)) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(x, y, grad):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = b.serve(x)[4]
                dw, db = mc2.mc2_matmul_weight_grad_quant(x, *mc2.mc2_act_quant(x))
            s.synchronize()
            if not (torch.equal(got, y) and torch.equal(dw, grad[0]) and torch.equal(db, grad[1])):
                bad.append(x.shape)

    threads = [threading.Thread(target=work, args=a) for a in zip(xs, want, grads)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and mc2.mc2_device_status() == mc2.MC2_OK


@pytest.mark.parametrize("m", [2, 100, 2500])
def test_with_a_stream_of_its_own(m):
    """``stream=``: workspaces and outputs come from that stream's pool, what the current stream allocates meanwhile is other memory."""
    b = Mlp(512, 1024)
    x = torch.randn(m, 512, generator=torch.Generator().manual_seed(0)).to(B).cuda()
    kept = mc2.mc2_act_quant(x, quant_mode=GROUP)
    want, grad = b.serve(x)[4], mc2.mc2_matmul_weight_grad_quant(x, *kept)
    vals, dz = mc2.mc2_act_dequant(*kept), mc2.mc2_act_grad_quant(x, *kept, activation="silu")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = b.serve(x, stream=s)[4]
    dw, db = mc2.mc2_matmul_weight_grad_quant(x, *kept, stream=s)
    v2, dz2 = mc2.mc2_act_dequant(*kept, stream=s), mc2.mc2_act_grad_quant(x, *kept, activation="silu", stream=s)
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (m * 512 * 2, m * 1024 * 2, 512 * 512 * 4, m * 512, 1 << 22) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in mine)
    assert torch.equal(got, want) and torch.equal(dw, grad[0]) and torch.equal(db, grad[1]) and torch.equal(v2, vals) and torch.equal(dz2, dz)


def slices(t):
    """The rows of t as a (3, m / 3, h) tensor of one stride, which the binding's extension module leaves to the Python code."""
    m, h = t.shape
    wide = torch.zeros(3, m // 3, h + 16, dtype=t.dtype, device=t.device)
    wide[:, :, :h] = t.view(3, m // 3, h)
    return wide[:, :, :h]


def test_both_marshalling_paths_agree():
    g = torch.Generator().manual_seed(0)
    z, dy = torch.randn(12, 256, generator=g).to(B).cuda(), torch.randn(12, 72, generator=g).to(B).cuda()
    w, ws = mc2.mc2_act_quant(torch.randn(72, 256, generator=g).cuda())
    for mode, kind in ((TOKEN, torch.int8), (GROUP, torch.float8_e4m3fn), (MX, torch.float8_e5m2)):
        q, s = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind, activation="silu")
        q3, s3 = mc2.mc2_act_quant(slices(z), quant_mode=mode, q_dtype=kind, activation="silu")
        assert torch.equal(q.view(torch.uint8).view(-1), q3.view(torch.uint8).view(-1)) and torch.equal(s.view(-1), s3.view(-1))
        out = mc2.mc2_act_dequant(q, s)
        wide = slices(torch.zeros_like(out))
        assert mc2.mc2_act_dequant(q3, s3, out=wide) is wide and torch.equal(wide.reshape(12, 256), out)
        a = mc2.mc2_act_grad_quant(z, q, s, activation="gelu")
        assert torch.equal(a.view(-1), mc2.mc2_act_grad_quant(slices(z), q3, s3, activation="gelu").view(-1))
        dw, db = mc2.mc2_matmul_weight_grad_quant(dy, q, s)
        dw3, db3 = mc2.mc2_matmul_weight_grad_quant(slices(dy), q3, s3)
        assert torch.equal(dw, dw3) and torch.equal(db, db3)
        if mode == TOKEN:
            y = mc2.mc2_quant_matmul(q, s, w, ws, residual=dy, activation="relu")
            y3 = mc2.mc2_quant_matmul(slices(q), s3, w, ws, residual=slices(dy), activation="relu")
            assert torch.equal(y.view(-1), y3.view(-1))


def test_given_outputs_and_workspaces_are_used():
    g = torch.Generator().manual_seed(1)
    z = torch.randn(1100, 256, generator=g).to(B).cuda()
    q, s = torch.empty(1100, 256, dtype=torch.int8, device="cuda"), torch.empty(1100, device="cuda")
    r = mc2.mc2_act_quant(z, q=q, scale=s)
    assert r[0] is q and r[1] is s
    w, ws = mc2.mc2_act_quant(torch.randn(2000, 256, generator=g).cuda())
    out = torch.empty(1100, 2000, dtype=torch.float16, device="cuda")
    size = mc2.mc2_quant_matmul_workspace(q, w, out)
    work = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    assert mc2.mc2_quant_matmul(q, s, w, ws, out=out, workspace=work) is out
    assert torch.equal(out, mc2.mc2_quant_matmul(q, s, w, ws, dtype=torch.float16))
    dw, db = torch.empty(256, 256, dtype=B, device="cuda"), torch.empty(256, dtype=B, device="cuda")
    work = torch.empty(mc2.mc2_matmul_weight_grad_quant_workspace(z, 256, dw=dw), dtype=torch.uint8, device="cuda")
    r = mc2.mc2_matmul_weight_grad_quant(z, q, s, dw=dw, db=db, workspace=work)
    want = mc2.mc2_matmul_weight_grad_quant(z, q, s)
    assert r[0] is dw and r[1] is db and torch.equal(dw, want[0]) and torch.equal(db, want[1])
    with pytest.raises(mc2.Mc2Error) as e:
        mc2.mc2_matmul_weight_grad_quant(z, q, s, workspace=work[:1024])
    assert e.value.status == mc2.MC2_ERR_WORKSPACE


def test_refusals():
    g = torch.Generator().manual_seed(0)
    z = torch.randn(4, 64, generator=g).to(B).cuda()
    q, s = mc2.mc2_act_quant(z)
    w, ws = mc2.mc2_act_quant(torch.randn(32, 64, generator=g).cuda())
    for f, match in ((lambda: mc2.mc2_quant_matmul(q.cpu(), s, w, ws), "x must be a CUDA tensor"),
                     (lambda: mc2.mc2_quant_matmul(q, s[:3], w, ws), "x_scale must have shape"),
                     (lambda: mc2.mc2_quant_matmul(q, s, w.t(), ws), "w must have shape"),
                     (lambda: mc2.mc2_quant_matmul(q, s, w, ws, bias=ws.half()), "bias must be of dtype"),
                     (lambda: mc2.mc2_quant_matmul(q, s, w, ws, activation="tanh"), "activation must be one of"),
                     (lambda: mc2.mc2_act_quant(z, q_dtype=torch.int32), "q_dtype must be"),
                     (lambda: mc2.mc2_act_dequant(z, s), "q must be of dtype"),
                     (lambda: mc2.mc2_act_dequant(q, s.view(4, 1).expand(4, 2)), "scale must have shape"),
                     (lambda: mc2.mc2_act_grad_quant(z[:3], q, s, activation="relu"), "dy must have shape"),
                     (lambda: mc2.mc2_matmul_weight_grad_quant(z[:3], q, s), "dy must have shape")):
        with pytest.raises(ValueError, match=match):
            f()
    for f, status in ((lambda: mc2.mc2_quant_matmul(q[:0], s[:0], w, ws), mc2.MC2_ERR_SHAPE),
                      (lambda: mc2.mc2_quant_matmul(q, s, w, ws, dtype=torch.float32), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_act_quant(z[:0]), mc2.MC2_ERR_SHAPE),
                      (lambda: mc2.mc2_act_quant(z, quant_mode=3), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_act_quant(z, quant_mode=MX), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_act_dequant(q, torch.zeros(4, 2, dtype=torch.uint8, device="cuda")), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_act_grad_quant(z.float(), q, s, activation="relu"), mc2.MC2_ERR_DTYPE),
                      (lambda: mc2.mc2_matmul_weight_grad_quant(z.float(), q, s), mc2.MC2_ERR_DTYPE)):
        with pytest.raises(mc2.Mc2Error) as e:
            f()
        assert e.value.status == status and e.value.message


def test_launch_events():
    """A call's kernels between the events installed for it."""
    z = torch.randn(300, 512, device="cuda").to(B)
    q, s = mc2.mc2_act_quant(z)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    for e in events:
        e.record()
    torch.cuda.synchronize()
    mc2.mc2_set_launch_events(events)
    try:
        mc2.mc2_matmul_weight_grad_quant(z, q, s)   # the values, the parts or the product, their sum
    finally:
        mc2.mc2_set_launch_events(None)
    torch.cuda.synchronize()
    assert events[0].elapsed_time(events[1]) > 0 and events[1].elapsed_time(events[2]) > 0
