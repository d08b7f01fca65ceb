"""mc2_matmul_bias_act, mc2_matmul_act_grad and mc2_act_grad against a plain
implementation in 64 bits.

Bounds.  A product of k terms is summed in fp32 (the tensor cores take 16 terms
a step): its error is below (k/16 + 16) 2^-23 S, S the sum of the terms' sizes.
(The plain kernel adds term by term, to nearest: k 2^-24 S.)  The activations'
slopes are below 1.2, and their own fp32 error below 2^-18 (1 + |z|); so an
output is within 1.2 times the product's bound, the activation's, and one
rounding to the type (2^-8 bf16, 2^-11 fp16, relative).
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
LEAST = {BF16: 1e-38, F16: 2.0 ** -25}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
OWN_ACT = 2.0 ** -18


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


def plain_derivative(z, act):
    if act == "relu":   # (clamp's own gradient is 1 at the bound itself; relu's is 0 at 0)
        return (z > 0).double()
    z = z.double().clone().requires_grad_()
    plain_act(z, act).sum().backward()
    return z.grad


def cut(t, wide):
    if not wide:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + wide), 3.0, dtype=t.dtype)
    big[:, :t.shape[1]] = t
    return big.cuda()[:, :t.shape[1]]


def make(m, n, k, dtype, seed, w_is_nk=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    x = cut(torch.randn(m, k, generator=g).to(dtype), wide)
    w = (torch.randn(n, k, generator=g) * k ** -0.5).to(dtype)
    w = cut(w if w_is_nk else w.t().contiguous(), wide)
    bias = (torch.randn(n, generator=g) * 0.3).to(dtype).cuda()
    res = cut(torch.randn(m, n, generator=g).to(dtype), wide)
    return x, w, bias, res


def product(x, w, w_is_nk):
    w64 = w.double().t() if w_is_nk else w.double()
    return x.double() @ w64, x.double().abs() @ w64.abs()


def acc_bound(k, size):
    return (k / 16 + 16) * 2.0 ** -23 * size


def within(got, ref, bound, what):
    assert got.shape == ref.shape
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d / bound).max()):.3g} of the bound"


def check_forward(m, n, k, dtype, act, use_bias, use_res, use_pre, w_is_nk, wide=0, seed=0):
    x, w, bias, res = make(m, n, k, dtype, seed, w_is_nk, wide)
    z, size = product(x, w, w_is_nk)
    if use_bias:
        z = z + bias.double()
    acc = acc_bound(k, size) + 2.0 ** -24 * z.abs()
    ref = plain_act(z, act)
    if use_res:
        ref = ref + res.double()
    out, pre = mc2.mc2_matmul_bias_act(x, w, w_is_nk=w_is_nk, bias=bias if use_bias else None, activation=act,
                                       residual=res if use_res else None, with_preact=use_pre)
    what = f"m={m} n={n} k={k} {dtype} {act} nk={w_is_nk}"
    within(out, ref, 1.2 * acc + (OWN_ACT * (1 + z.abs()) if act != "none" else 0) + 2.0 ** -24 * ref.abs() +
           UNIT[dtype] * ref.abs() + LEAST[dtype], what + " out")
    if use_pre:
        within(pre, z, acc + UNIT[dtype] * z.abs() + LEAST[dtype], what + " preact")
    else:
        assert pre is None


# sizes around the tiles' edges (16, 32, 64, 128, 256 rows; 64 and 128 columns; 64-deep steps), the smallest, odd
# ones, and some that leave most of a wave empty or fill several
SIZES = [(1, 8, 8), (1, 1, 1), (1, 4096, 4096), (2, 136, 64), (7, 128, 72), (15, 1000, 1000), (16, 64, 128),
         (17, 72, 2056), (24, 512, 8192), (31, 256, 256), (33, 264, 1040), (63, 128, 512), (64, 1024, 1024),
         (65, 200, 320), (100, 5000, 96), (127, 136, 1000), (128, 256, 2048), (129, 512, 512), (200, 1000, 4096),
         (255, 384, 640), (256, 256, 1024), (257, 264, 136), (300, 2048, 8), (520, 1000, 264), (777, 1000, 2056),
         (1100, 1104, 1032), (2100, 96, 128), (1500, 2600, 64), (4096, 512, 256), (128, 10000, 4160),
         (250, 5000, 4096), (60, 40000, 5000), (700, 512, 16384), (2000, 1024, 24576)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_forward_sizes(m, n, k, w_is_nk):
    i = SIZES.index((m, n, k)) + (0 if w_is_nk else 1)
    check_forward(m, n, k, BF16 if i % 2 else F16, ACTS[i % 5], i % 3 != 0, i % 2 == 0, i % 4 == 1, w_is_nk, seed=i)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("use_bias,use_res,use_pre", [(False, False, False), (True, False, False), (False, True, False),
                                                      (True, True, True), (True, False, True)])
@pytest.mark.parametrize("m,n,k", [(3, 256, 512), (90, 192, 256), (1040, 520, 192)])
def test_forward_epilogues(m, n, k, act, use_bias, use_res, use_pre):
    check_forward(m, n, k, BF16, act, use_bias, use_res, use_pre, True, seed=m)


@pytest.mark.parametrize("m,n,k,wide", [(5, 33, 65, 0), (5, 128, 100, 0), (70, 77, 128, 0), (130, 129, 67, 3),
                                        (9, 136, 200, 8), (300, 72, 264, 24), (700, 1001, 333, 7), (1, 513, 1027, 5)])
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_odd_sizes_and_strides(m, n, k, wide, w_is_nk):
    check_forward(m, n, k, F16, "gelu_tanh", True, True, True, w_is_nk, wide=wide, seed=n)


@pytest.mark.parametrize("m,n,k", [(4, 77, 40), (200, 77, 40), (900, 333, 136)])
def test_odd_widths_in_aligned_rows(m, n, k):
    """n odd in rows of a stride that is a multiple of 8: written to the last column, not past it."""
    x, w, bias, _ = make(m, n, k, BF16, seed=5)
    wide = torch.full((m, n + (-n % 8) + 8), 9.0, dtype=BF16, device="cuda")
    out, _ = mc2.mc2_matmul_bias_act(x, w, bias=bias, out=wide[:, :n])
    z, size = product(x, w, True)
    z = z + bias.double()
    within(out, z, acc_bound(k, size) + UNIT[BF16] * z.abs() + 2.0 ** -23 * z.abs() + 1e-38, "out")
    assert (wide[:, n:] == 9).all()


@pytest.mark.parametrize("m,n,k", [(1, 72, 67), (40, 136, 131), (500, 264, 1021), (1300, 77, 5), (2100, 1100, 77)])
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_odd_depths_in_aligned_rows(m, n, k, w_is_nk):
    """k (and n) odd in rows of a stride that is a multiple of 8: what lies between a row's end
    and the next row's start (here NaN) enters no sum."""
    def padded(t):
        big = torch.full((t.shape[0], t.shape[1] + (-t.shape[1] % 8) + 8), float("nan"), dtype=t.dtype, device="cuda")
        big[:, :t.shape[1]] = t
        return big[:, :t.shape[1]]

    x, w, bias, res = make(m, n, k, BF16, 6, w_is_nk)
    z, size = product(x, w, w_is_nk)
    z = z + bias.double()
    ref = plain_act(z, "silu") + res.double()
    out, pre = mc2.mc2_matmul_bias_act(padded(x), padded(w), w_is_nk=w_is_nk, bias=bias, activation="silu",
                                       residual=padded(res), with_preact=True)
    within(pre, z, acc_bound(k, size) + UNIT[BF16] * z.abs() + 2.0 ** -23 * z.abs() + 1e-38, "preact")
    within(out, ref, 1.2 * acc_bound(k, size) + OWN_ACT * (1 + z.abs()) + (UNIT[BF16] + 2.0 ** -22) * ref.abs() + 1e-38, "out")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("w_is_nk", [True, False])
@pytest.mark.parametrize("m,n,k", [(1, 264, 1040), (20, 520, 712), (140, 136, 328), (1090, 272, 328), (350, 1000, 72)])
def test_integer_values_bit_exact(m, n, k, w_is_nk, dtype):
    """Small integers: every sum is exact in fp32 and every output in 16 bits, so
    a shifted, dropped or doubled term shows in any bit."""
    g = torch.Generator().manual_seed(m)
    x = torch.randint(-2, 3, (m, k), generator=g).to(dtype).cuda()
    w = (torch.randint(-2, 3, (n, k), generator=g) * (torch.rand(n, k, generator=g) < 0.1)).to(dtype)
    w = (w if w_is_nk else w.t().contiguous()).cuda()
    bias = torch.randint(-3, 4, (n,), generator=g).to(dtype).cuda()
    res = torch.randint(-4, 5, (m, n), generator=g).to(dtype).cuda()
    z = product(x, w, w_is_nk)[0] + bias.double()
    assert float(z.abs().max()) <= 240
    out, pre = mc2.mc2_matmul_bias_act(x, w, w_is_nk=w_is_nk, bias=bias, activation="relu", residual=res, with_preact=True)
    assert torch.equal(pre.double(), z)
    assert torch.equal(out.double(), z.clamp(min=0) + res.double())


def test_residual_in_place_three_dimensions_and_a_side_stream():
    for m3, n, k in (((2, 3), 256, 320), ((5, 100), 520, 192)):
        m = m3[0] * m3[1]
        x, w, bias, res = make(m, n, k, BF16, seed=4)
        ref = plain_act(product(x, w, True)[0] + bias.double(), "silu") + res.double()
        size = product(x, w, True)[1]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        r3 = res.view(*m3, n)
        out, _ = mc2.mc2_matmul_bias_act(x.view(*m3, k), w, bias=bias, activation="silu", residual=r3, out=r3, stream=s)
        s.synchronize()
        assert out.data_ptr() == res.data_ptr() and out.shape == (*m3, n)
        within(out.view(m, n), ref, 1.2 * acc_bound(k, size) + OWN_ACT * (1 + ref.abs()) * 2 + UNIT[BF16] * ref.abs(), "in place")


def test_nan_and_infinity_stay_in_their_rows():
    for m in (6, 400):
        x, w, _, _ = make(m, 136, 200, BF16, seed=1)
        clean, _ = mc2.mc2_matmul_bias_act(x, w)
        x[2, 5] = float("nan")
        x[4, 199] = float("inf")
        got, _ = mc2.mc2_matmul_bias_act(x, w)
        assert got[2].isnan().all()
        assert not got[4].isfinite().any()
        keep = [i for i in range(m) if i not in (2, 4)]
        assert torch.equal(got[keep], clean[keep])
        relu, _ = mc2.mc2_matmul_bias_act(x, w, activation="relu")
        assert relu[2].isnan().all()


@pytest.mark.parametrize("m", [3, 90, 700])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_a_nan_or_infinity_stays_in_its_element(m, act):
    """One column of the bias, one element of z: the columns beside it are as without it."""
    x, w, bias, _ = make(m, 136, 64, BF16, seed=2)
    clean, _ = mc2.mc2_matmul_bias_act(x, w, bias=bias, activation=act)
    for bad in (float("nan"), float("inf"), -float("inf")):
        b = bias.clone()
        b[17] = bad
        got, _ = mc2.mc2_matmul_bias_act(x, w, bias=b, activation=act)
        keep = [i for i in range(136) if i != 17]
        assert torch.equal(got[:, keep], clean[:, keep])
        if bad != bad:
            assert got[:, 17].isnan().all()
        elif bad > 0:
            assert (got[:, 17] == bad).all()
        else:
            assert (got[:, 17].abs() < 1e-15).all()   # the limit, 0
    z = (3 * torch.randn(m, 64, generator=torch.Generator().manual_seed(m))).to(BF16).cuda()
    dy = torch.randn(m, 136, generator=torch.Generator().manual_seed(m + 1)).to(BF16).cuda()
    clean = mc2.mc2_matmul_act_grad(dy, w, z, activation=act)
    z[m // 2, 8] = float("nan")
    got = mc2.mc2_matmul_act_grad(dy, w, z, activation=act)
    assert got[m // 2, 8].isnan()
    got[m // 2, 8] = clean[m // 2, 8]
    assert torch.equal(got, clean)


def test_same_bits_every_time():
    for m, n, k in ((1, 4096, 4096), (40, 1024, 8192), (333, 1000, 2056)):
        x, w, bias, res = make(m, n, k, BF16, seed=7)
        a, _ = mc2.mc2_matmul_bias_act(x, w, bias=bias, activation="gelu", residual=res)
        b, _ = mc2.mc2_matmul_bias_act(x, w, bias=bias, activation="gelu", residual=res)
        assert torch.equal(a, b)


def test_launches_beside_one_another():
    """Shapes with one and two CTAs an SM, pairs and clusters, on streams of their own: the bits of a call by itself."""
    cases = []
    for i, (m, n, k) in enumerate(((1, 4096, 4096), (16, 1000, 2056), (32, 1024, 8192), (64, 4096, 512), (128, 1024, 4096),
                                   (300, 4096, 1024), (512, 1000, 2056), (777, 2048, 512))):
        x, w, bias, res = make(m, n, k, BF16 if i % 2 else F16, seed=i)
        cases.append((x, w, bias, res, mc2.mc2_matmul_bias_act(x, w, bias=bias, activation="silu", residual=res)[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i in range(240):
        x, w, bias, res, want = cases[(5 * i + i // 8) % 8]
        with torch.cuda.stream(streams[i % 4]):
            got.append((mc2.mc2_matmul_bias_act(x, w, bias=bias, activation="silu", residual=res)[0], want))
    torch.cuda.synchronize()
    assert mc2.mc2_device_status() == mc2.MC2_OK
    assert all(torch.equal(o, want) for o, want in got)


# ------------------------------------------------------------------ gradients

def check_act_grad(m, n, k, dtype, act, w_is_nk, wide=0, seed=0, in_place=False):
    g = torch.Generator().manual_seed(seed)
    dy = cut(torch.randn(m, n, generator=g).to(dtype), wide)
    w = (torch.randn(n, k, generator=g) * n ** -0.5).to(dtype)
    w = cut(w if w_is_nk else w.t().contiguous(), wide)
    z = cut((2 * torch.randn(m, k, generator=g)).to(dtype), wide)
    w64 = w.double() if w_is_nk else w.double().t()
    dx, size = dy.double() @ w64, dy.double().abs() @ w64.abs()
    d = plain_derivative(z, act)
    ref = dx * d
    # (1 + |z|) 2^-18 bounds the derivative's fp32 error
    bound = acc_bound(n, size) * 1.2 + OWN_ACT * (1 + z.double().abs()) * dx.abs() * (act != "relu") + \
        (UNIT[dtype] + 2.0 ** -23) * ref.abs() + LEAST[dtype]
    got = mc2.mc2_matmul_act_grad(dy, w, z, activation=act, w_is_nk=w_is_nk, dz=z if in_place else None)
    within(got, ref, bound, f"m={m} n={n} k={k} {act}")


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_act_grad_sizes(m, n, k, w_is_nk):
    i = SIZES.index((m, n, k))
    check_act_grad(m, n, k, F16 if i % 2 else BF16, ACTS[1 + i % 4], w_is_nk, seed=i, in_place=i % 3 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,wide", [(5, 96, 256, 0), (600, 320, 264, 0), (77, 33, 129, 1)])
def test_act_grad_activations(act, m, n, k, wide):
    check_act_grad(m, n, k, BF16, act, True, wide=wide, seed=m)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,wide", [(1, 1, 0), (3, 1000, 0), (129, 257, 0), (64, 512, 8), (1000, 2049, 3)])
def test_elementwise_act_grad(act, m, n, wide):
    g = torch.Generator().manual_seed(m + n)
    for dtype in (BF16, F16):
        dy = cut(torch.randn(m, n, generator=g).to(dtype), wide)
        z = cut((3 * torch.randn(m, n, generator=g)).to(dtype), wide)
        ref = dy.double() * plain_derivative(z, act)
        got = mc2.mc2_act_grad(dy, z, activation=act)
        within(got, ref, OWN_ACT * (1 + z.double().abs()) * dy.double().abs() * (act != "relu") +
               (UNIT[dtype] + 2.0 ** -23) * ref.abs() + LEAST[dtype], f"{act} {dtype}")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_derivative_at_its_limits(act):
    """Far from zero the derivative is its limit, at infinity too; a NaN stays one."""
    z = torch.tensor([[-float("inf"), -6e4, -100.0, 100.0, 6e4, float("inf"), float("nan"), 0.0]], dtype=F16).cuda()
    dy = torch.full_like(z, 2.0)
    got = mc2.mc2_act_grad(dy, z, activation=act)[0].tolist()
    assert got[:3] == [0, 0, 0] and got[3:6] == [2, 2, 2] and got[6] != got[6] and got[7] == 1.0


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_relu_derivative_at_zero(dtype):
    """1 above zero down to the least number of the type, 0 at both zeros and below, in each form of the call."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    row = torch.tensor([0.0, -0.0, tiny, -tiny, 1.0, -1.0, float("inf"), -float("inf")], dtype=dtype)
    want = [0, 0, 1, 0, 1, 0, 1, 0]
    for m in (2, 300, 2000):
        z = row.repeat(m, 1).cuda()
        one = torch.ones(m, 8, dtype=dtype, device="cuda")
        w = torch.full((8, 8), 0.125, dtype=dtype, device="cuda")   # one @ w is 1 everywhere
        wide = torch.zeros(m, 9, dtype=dtype, device="cuda")       # rows that the plain kernels take
        wide[:, :8] = z
        for at in (z, wide[:, :8]):
            assert mc2.mc2_act_grad(one, at, activation="relu")[m - 1].tolist() == want
            assert mc2.mc2_matmul_act_grad(one, w, at, activation="relu")[m - 1].tolist() == want


def test_derivatives_against_differences():
    """Central differences of the 64-bit activations at step 1e-5: an error near
    1e-10, far below the fp16 output's 2^-11."""
    z = torch.linspace(-8, 8, 4001, dtype=torch.float64).to(F16).view(1, -1).cuda()
    dy = torch.ones_like(z)
    for act in ("gelu", "gelu_tanh", "silu"):
        t = 1e-5
        slope = (plain_act(z.double() + t, act) - plain_act(z.double() - t, act)) / (2 * t)
        got = mc2.mc2_act_grad(dy, z, activation=act)
        within(got, slope, OWN_ACT * (1 + z.double().abs()) + UNIT[F16] * slope.abs() + LEAST[F16] + 1e-9, act)


@pytest.mark.parametrize("m,d,f", [(5, 256, 512), (300, 264, 520)])
def test_a_block_forward_and_backward(m, d, f):
    """The calls together: y = x2 + W2 act(W1 norm(x + r) + b1) + b2 and all its gradients against autograd in
    64 bits.  Each 16-bit tensor in between is rounded once, so gradients agree to a few 2^-8 of their size."""
    g = torch.Generator().manual_seed(m)

    def t(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(BF16).cuda()

    x, r, wn = t(m, d), t(m, d), (1 + 0.1 * t(d)).to(BF16)
    w1, b1, w2, b2, dy = t(f, d, std=d ** -0.5), t(f, std=0.1), t(d, f, std=f ** -0.5), t(d, std=0.1), t(m, d, std=0.1)
    nrm = mc2.mc2_add_rms_norm(x, wn, residual=r, with_rstd=True)
    h, z = mc2.mc2_matmul_bias_act(nrm["out"], w1, bias=b1, activation="gelu_tanh", with_preact=True)
    y, _ = mc2.mc2_matmul_bias_act(h, w2, bias=b2, residual=nrm["residual"])
    dz = mc2.mc2_matmul_act_grad(dy, w2, z, activation="gelu_tanh")
    dw2, db2 = mc2.mc2_matmul_weight_grad(dy, h)
    dw1, db1 = mc2.mc2_matmul_weight_grad(dz, nrm["out"])
    dn, _ = mc2.mc2_matmul_bias_act(dz, w1, w_is_nk=False)
    dx, dwn = mc2.mc2_rms_norm_grad(dn, nrm["residual"], wn, nrm["rstd"], dres=dy)

    p = [v.double().requires_grad_() for v in (x, wn, w1, b1, w2, b2)]
    s = p[0] + r.double()
    n64 = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * p[1]
    y64 = plain_act(n64 @ p[2].t() + p[3], "gelu_tanh") @ p[4].t() + p[5] + s
    y64.backward(dy.double())
    for got, ref, what in ((y, y64.detach(), "y"), (dx, p[0].grad, "dx"), (dwn, p[1].grad, "dwn"), (dw1, p[2].grad, "dw1"),
                           (db1, p[3].grad, "db1"), (dw2, p[4].grad, "dw2"), (db2, p[5].grad, "db2")):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= 3 * UNIT[BF16], (what, rel)
