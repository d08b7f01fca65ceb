"""mc2_matmul_weight_grad_quant against a plain implementation in 64 bits.

Bounds.  A term dy a, a = act(q scale), has the rounding of a to the operands' type (2^-8 bf16, 2^-11 fp16, relative; none
where a is a code times a power of two) and, with an activation, a's own fp32 error, below 2^-18 (1 + |z|).  Sums of m terms are fp32 (16 terms
a step of the tensor cores): (m / 16 + 16) 2^-23 of the terms' sizes; dw is rounded once.  db is summed term by term, to
nearest: m 2^-24 of the terms' sizes, and one rounding.
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
I8, E4M3, E5M2 = torch.int8, torch.float8_e4m3fn, torch.float8_e5m2
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
LEAST = {BF16: 1e-38, F16: 2.0 ** -25}
QMAX = {I8: 127.0, E4M3: 448.0, E5M2: 57344.0}
TOKEN, GROUP, MX = mc2.QUANT_PERTOKEN_DYNAMIC, mc2.QUANT_PERGROUP, mc2.QUANT_MX
KINDS = [(TOKEN, I8), (TOKEN, E4M3), (TOKEN, E5M2), (GROUP, I8), (GROUP, E4M3), (GROUP, E5M2), (MX, E4M3), (MX, E5M2)]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def plain_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.erfc(-z * 0.5 ** 0.5) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def cut(t, wide):
    if not wide:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + wide), 3.0, dtype=t.dtype)
    big[:, 1:1 + t.shape[1]] = t
    return big.cuda()[:, 1:1 + t.shape[1]]


def kept(m, k, mode, kind, g):
    """Codes of normal values with scales that bring them to a size near one, made without the library."""
    v = torch.randn(m, k, generator=g)
    if kind == I8:
        q = (v * 40).round().clamp(-127, 127).to(I8)
        scale = (torch.rand(m, generator=g) if mode == TOKEN else torch.rand(m, -(-k // 128), generator=g)) / 32
    else:
        q = (v * (100 if kind == E4M3 else 16000)).clamp(-QMAX[kind], QMAX[kind]).to(kind)
        unit = 2.0 ** -7 if kind == E4M3 else 2.0 ** -14
        if mode == MX:
            scale = (torch.randint(-2, 2, (m, -(-k // 32)), generator=g) + (120 if kind == E4M3 else 113)).to(torch.uint8)
        else:
            scale = (torch.rand(m, generator=g) if mode == TOKEN else torch.rand(m, -(-k // 128), generator=g)) * unit
    return q.cuda(), scale.cuda()


def values(q, scale, mode):
    k = q.shape[1]
    s = scale.double() if mode != MX else torch.ldexp(torch.ones_like(scale, dtype=torch.float64), scale.int() - 127)
    return q.double() * s.view(s.shape[0], -1).repeat_interleave({TOKEN: k, GROUP: 128, MX: 32}[mode], 1)[:, :k]


def check(m, n, k, dtype, act, mode, kind, wide=0, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    q, scale = kept(m, k, mode, kind, g)
    dy = cut((torch.randn(m, n, generator=g) * 0.1).to(dtype), wide)
    dw, db = mc2.mc2_matmul_weight_grad_quant(dy, q, scale, activation=act, **kw)
    assert dw.shape == (n, k) and dw.dtype == dtype and db.shape == (n,) and db.dtype == dtype
    z, d = values(q, scale, mode), dy.double()
    a = plain_act(z, act)
    ref, size = d.t() @ a, d.abs().t() @ a.abs()
    per = (UNIT[dtype] + 2.0 ** -23) * a.abs() + LEAST[dtype]
    if act != "none":
        per = per + (2.0 ** -18 + 1.2 * 2.0 ** -24) * (1 + z.abs())
    bound = d.abs().t() @ per + (m / 16 + 16) * 2.0 ** -23 * size + UNIT[dtype] * ref.abs() + LEAST[dtype]
    bad = ~((dw.double() - ref).abs() <= bound)
    assert not bad.any(), f"m={m} n={n} k={k} {dtype} {act} {mode} {kind}: {int(bad.sum())} of {bad.numel()} outside"
    # the bound's own size: a wrong scale or a lost token stands out of the rounding's 2-norm
    off = float((dw.double() - ref).norm() / ref.norm().clamp(min=1e-30))
    assert off <= 1.5 * UNIT[dtype] + 2.0 ** -12, off
    want, size = d.sum(0), d.abs().sum(0)
    assert ((db.double() - want).abs() <= m * 2.0 ** -24 * size + UNIT[dtype] * want.abs() + LEAST[dtype]).all()
    return dw, db, (dy, q, scale)


SIZES = [(1, 1, 1), (1, 64, 128), (2, 8, 8), (3, 130, 65), (16, 256, 256), (63, 257, 255), (64, 128, 64), (65, 100, 1000), (130, 1000, 136),
         (197, 72, 4104), (333, 1000, 1001), (1000, 512, 512), (1025, 300, 200), (2048, 256, 2048), (4100, 136, 264), (20000, 64, 72),
         (16384, 512, 256), (500, 4096, 96), (300, 2600, 2600)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("which", range(4))
def test_sizes(m, n, k, which):
    i = SIZES.index((m, n, k)) * 3 + which
    mode, kind = KINDS[i % 8]
    check(m, n, k, BF16 if i % 2 else F16, ACTS[i % 5], mode, kind, seed=i)


@pytest.mark.parametrize("mode,kind", KINDS)
@pytest.mark.parametrize("act", ACTS)
def test_codes_and_activations(mode, kind, act):
    for dtype in (BF16, F16):
        check(150, 136, 328, dtype, act, mode, kind, seed=5)


@pytest.mark.parametrize("m,n,k", [(70, 200, 300), (300, 264, 512), (5, 33, 47), (3000, 130, 100)])
@pytest.mark.parametrize("wide", [1, 8, 9])
def test_strided_rows_of_dy(m, n, k, wide):
    check(m, n, k, BF16, "none", GROUP, I8, wide=wide, seed=2)


@pytest.mark.parametrize("m,n,k", [(300, 264, 512), (5, 33, 47), (9000, 130, 104)])
def test_given_outputs_and_alignments(m, n, k):
    """Outputs of one's own, at any element's address, and without the bias gradient."""
    dw, db, (dy, q, scale) = check(m, n, k, BF16, "silu", TOKEN, I8, seed=4)
    for shift in (0, 1, 8):
        a = torch.full((n * k + 16,), 7.0, dtype=BF16, device="cuda")
        b = torch.full((n + 16,), 7.0, dtype=BF16, device="cuda")
        w, v = a[shift:shift + n * k].view(n, k), b[shift:shift + n]
        r = mc2.mc2_matmul_weight_grad_quant(dy, q, scale, activation="silu", dw=w, db=v)
        assert r[0] is w and r[1] is v
        assert (w.double() - dw.double()).norm() <= 2.0 ** -8 * dw.double().norm()
        assert (v.double() - db.double()).norm() <= 2.0 ** -8 * db.double().norm()
        assert (a[:shift] == 7).all() and (a[shift + n * k:] == 7).all() and (b[:shift] == 7).all() and (b[shift + n:] == 7).all()
    again, none = mc2.mc2_matmul_weight_grad_quant(dy, q, scale, activation="silu", with_bias=False)
    assert none is None and torch.equal(again, dw)


def test_against_differences():
    """L = sum(y g) with y = act(x) @ w^T: its difference in w is dw for dy = g, exactly linear, so one step will do."""
    g = torch.Generator().manual_seed(3)
    m, n, k = 96, 40, 72
    q, scale = kept(m, k, TOKEN, I8, g)
    grad = torch.randn(m, n, generator=g).to(F16).cuda()
    dw, db = mc2.mc2_matmul_weight_grad_quant(grad, q, scale, activation="gelu")
    a = plain_act(values(q, scale, TOKEN), "gelu")
    w = torch.randn(n, k, generator=g).double().cuda()
    for i, j in ((0, 0), (39, 71), (17, 30)):
        step = torch.zeros_like(w)
        step[i, j] = 0.5
        diff = ((a @ (w + step).t() - a @ (w - step).t()) * grad.double()).sum()
        size = (a[:, j].abs() * grad[:, i].double().abs()).sum()
        assert abs(float(dw[i, j]) - float(diff)) <= float(2.0 ** -10 * size) + 2.0 ** -11 * abs(float(diff))


def test_a_token_that_is_not_a_number():
    """Its group's columns are NaN, the others as without that group."""
    m, n, k = 140, 130, 384
    g = torch.Generator().manual_seed(1)
    q, scale = kept(m, k, GROUP, I8, g)
    dy = torch.randn(m, n, generator=g).to(BF16).cuda()
    clean, _ = mc2.mc2_matmul_weight_grad_quant(dy, q, scale)
    scale[7, 1] = float("nan")
    dw, db = mc2.mc2_matmul_weight_grad_quant(dy, q, scale)
    assert dw[:, 128:256].isnan().all() and torch.equal(dw[:, :128], clean[:, :128]) and torch.equal(dw[:, 256:], clean[:, 256:])
    assert db.isfinite().all()


def test_zero_tokens_change_nothing():
    """A padded batch: rows of zero gradients and of zero scales add nothing."""
    m, n, k = 200, 264, 520
    g = torch.Generator().manual_seed(6)
    q, scale = kept(m, k, TOKEN, I8, g)
    dy = torch.randn(m, n, generator=g).to(BF16).cuda()
    dy[100:] = 0
    a = mc2.mc2_matmul_weight_grad_quant(dy, q, scale)
    scale[150:] = 0
    b = mc2.mc2_matmul_weight_grad_quant(dy, q, scale)
    c = mc2.mc2_matmul_weight_grad_quant(dy[:100].contiguous(), q[:100].contiguous(), scale[:100].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0].double() - c[0].double()).norm() <= 2.0 ** -8 * c[0].double().norm()


def test_more_dimensions():
    g = torch.Generator().manual_seed(8)
    q, scale = kept(24, 128, GROUP, I8, g)
    dy = torch.randn(24, 64, generator=g).to(BF16).cuda()
    a = mc2.mc2_matmul_weight_grad_quant(dy, q, scale)
    b = mc2.mc2_matmul_weight_grad_quant(dy.view(2, 12, 64), q.view(2, 12, 128), scale.view(2, 12, 1))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
