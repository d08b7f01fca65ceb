"""mc2_quant_matmul against a plain implementation: the integer sums in 64 bits, then the header's fp32 steps.

Without an activation every step is one fp32 operation that rounds to nearest, so the result is compared bit for
bit: float(acc) x_scale, times w_scale, plus bias, plus residual, rounded to the type.  An activation's own fp32 error is
below 2^-18 (1 + |z|), its slope below 1.2 (z itself is then within 4 x 2^-24 of the 64-bit one, relative to the
product's and the bias's sizes), and the output is rounded once (2^-8 bf16, 2^-11 fp16, relative; 2^-25 absolute
for fp16's subnormals).
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
LEAST = {BF16: 1e-38, F16: 2.0 ** -25}
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
    """t, or t as a slice of a wider tensor: `wide` columns more, the first of them before it."""
    if not wide:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + wide), 3, dtype=t.dtype)
    big[:, 1:1 + t.shape[1]] = t
    return big.cuda()[:, 1:1 + t.shape[1]]


def make(m, n, k, seed, w_is_nk=True, wide=0, span=127):
    g = torch.Generator().manual_seed(seed)
    x = cut(torch.randint(-span, span + 1, (m, k), generator=g, dtype=torch.int8), wide)
    w = torch.randint(-span, span + 1, (n, k), generator=g, dtype=torch.int8)
    w = cut(w if w_is_nk else w.t().contiguous(), wide)
    # products of a size near one
    xs = (torch.rand(m, generator=g) + 0.5).cuda() / 4096
    ws = (torch.rand(n, generator=g) + 0.5).cuda() / (k ** 0.5)
    return x, xs, w, ws


def sums(x, w, w_is_nk):
    """x @ w^T exactly: fp64 holds these integers."""
    return x.double() @ (w.double().t() if w_is_nk else w.double())


def check(m, n, k, dtype, act, bias_type, use_res, w_is_nk, wide=0, seed=0):
    x, xs, w, ws = make(m, n, k, seed, w_is_nk, wide)
    g = torch.Generator().manual_seed(seed + 1)
    bias = None if bias_type is None else (torch.randn(n, generator=g) * 0.3).to(bias_type).cuda()
    res = cut(torch.randn(m, n, generator=g).to(dtype), wide) if use_res else None
    out = mc2.mc2_quant_matmul(x, xs, w, ws, w_is_nk=w_is_nk, bias=bias, activation=act, residual=res, dtype=dtype)
    assert out.shape == (m, n) and out.dtype == dtype
    acc = sums(x, w, w_is_nk)
    what = f"m={m} n={n} k={k} {dtype} {act} nk={w_is_nk} wide={wide}"
    if act == "none":
        z = acc.float() * xs[:, None] * ws
        if bias is not None:
            z = z + bias.float()
        if res is not None:
            z = z + res.float()
        bad = out != z.to(dtype)
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"
        return
    p = acc * xs.double()[:, None] * ws.double()
    z = p if bias is None else p + bias.double()
    ref = plain_act(z, act)
    if res is not None:
        ref = ref + res.double()
    bound = 1.2 * 4 * 2.0 ** -24 * (p.abs() + z.abs()) + 2.0 ** -18 * (1 + z.abs()) + (UNIT[dtype] + 2.0 ** -24) * ref.abs() + LEAST[dtype]
    bad = ~((out.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


# sizes around the tiles' edges (16 to 256 tokens, 128 and 256 columns, 64, 128 and 1024 deep), the smallest, odd ones,
# and some that leave most of a wave empty or fill several
SIZES = [(1, 1, 1), (1, 8, 16), (1, 128, 128), (1, 4096, 4096), (1, 1000, 16384), (2, 136, 64), (3, 130, 129), (7, 128, 72),
         (15, 1000, 1008), (16, 64, 128), (17, 72, 2056), (24, 512, 8192), (31, 256, 256), (33, 264, 1040), (48, 4096, 1024),
         (63, 127, 511), (64, 1024, 1024), (65, 200, 320), (100, 5000, 96), (127, 136, 1000), (128, 256, 2048), (129, 512, 512),
         (200, 1008, 4096), (255, 384, 640), (256, 256, 1024), (257, 264, 136), (300, 2048, 8), (520, 1000, 264),
         (777, 1000, 2056), (1100, 1104, 1040), (2100, 96, 128), (1500, 2600, 64), (4096, 512, 256), (128, 10000, 4160),
         (60, 40000, 512), (700, 512, 16384), (300, 513, 12289), (2000, 1024, 4096)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("w_is_nk", [True, False])
def test_sizes(m, n, k, w_is_nk):
    i = SIZES.index((m, n, k)) + (0 if w_is_nk else 1)
    check(m, n, k, BF16 if i % 2 else F16, "none", [None, BF16 if i % 2 else F16, torch.float32][i % 3], i % 2 == 0, w_is_nk, seed=i)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias_type,use_res", [(None, False), (BF16, False), (torch.float32, True)])
@pytest.mark.parametrize("m,n,k", [(3, 256, 512), (90, 192, 256), (1040, 520, 192)])
def test_epilogues(m, n, k, act, bias_type, use_res):
    check(m, n, k, BF16, act, bias_type, use_res, True, seed=3)


@pytest.mark.parametrize("m,n,k", [(1, 250, 333), (20, 144, 272), (130, 512, 1024), (900, 520, 250)])
@pytest.mark.parametrize("w_is_nk", [True, False])
@pytest.mark.parametrize("wide", [1, 16, 17])
def test_strides_and_alignments(m, n, k, w_is_nk, wide):
    check(m, n, k, F16, "none", torch.float32, True, w_is_nk, wide=wide, seed=wide)


@pytest.mark.parametrize("m", [1, 5, 40, 300])
@pytest.mark.parametrize("k", [1024, 1025, 5000, 33000])
def test_largest_codes(m, k):
    """All codes at an end of int8: the largest sums, and a product of ends of both signs."""
    n = 160
    w = torch.full((n, k), -128, dtype=torch.int8)
    w[::2] = 127
    x = torch.full((m, k), -128, dtype=torch.int8)
    x[::3] = 127
    x, w, one = x.cuda(), w.cuda(), torch.ones
    xs, ws = one(m, device="cuda") * 2.0 ** -30, one(n, device="cuda")
    out = mc2.mc2_quant_matmul(x, xs, w, ws, dtype=BF16)
    want = (sums(x, w, True).float() * 2.0 ** -30).to(BF16)
    assert torch.equal(out, want)


def test_the_deepest_product():
    """k = 131071, where sums of -128 times -128 come next to 2^31."""
    k = 131071
    x = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((20, k), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones
    for t in (x, x.repeat(100, 1)):
        out = mc2.mc2_quant_matmul(t, one(t.shape[0], device="cuda"), w, one(20, device="cuda"), dtype=BF16)
        assert torch.equal(out, sums(t, w, True).float().to(BF16))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,k", [(512, 4096), (1001, 2056), (333, 1000)])
@pytest.mark.parametrize("bias_type", [None, BF16, torch.float32])
def test_a_token_does_not_depend_on_the_others(n, k, act, bias_type):
    """The same bits for a row by itself, in a batch, and in a prompt; and from strided rows."""
    x, xs, w, ws = make(1200, n, k, 5)
    ws[::3] *= -1     # (negative zeros, too)
    x[5] = 0
    bias = None if bias_type is None else torch.randn(n, device="cuda").to(bias_type)

    def bits(rows, scales):
        return mc2.mc2_quant_matmul(rows, scales, w, ws, bias=bias, activation=act).view(torch.int16)

    whole = bits(x, xs)
    for m in (1, 2, 4, 7, 17, 64, 100, 250, 600):
        assert torch.equal(bits(x[:m], xs[:m]), whole[:m]), m
    for first in range(4, 1200, 149):
        assert torch.equal(bits(x[first:first + 4], xs[first:first + 4]), whole[first:first + 4]), first
    wide = torch.zeros(70, k + 5, dtype=torch.int8, device="cuda")
    wide[:, 3:3 + k] = x[:70]
    assert torch.equal(bits(wide[:, 3:3 + k], xs[:70]), whole[:70])


def test_scales_that_are_zero_or_not_numbers():
    """A zero row's scale is zero; a NaN or an infinity stays in its row (the codes there are zeros) or column."""
    m, n, k = 130, 260, 256
    for rows in (m, 5):
        x, xs, w, ws = make(rows, n, k, 9)
        xs[0], xs[1], xs[2] = 0.0, float("nan"), float("inf")
        x[1:3] = 0
        ws[7], ws[8] = 0.0, float("nan")
        out = mc2.mc2_quant_matmul(x, xs, w, ws, activation="gelu")
        clean = torch.ones(n, dtype=torch.bool, device="cuda")
        clean[8] = False
        assert (out[0, clean] == 0).all() and out[1:3].isnan().all() and out[:, 8].isnan().all()
        assert (out[3:, 7] == 0).all() and out[3:, clean].isfinite().all()


def test_the_residual_in_place_and_rows_after_the_last():
    m, n, k = 200, 264, 512
    for rows in (m, 9):
        x, xs, w, ws = make(rows, n, k, 11)
        big = torch.randn(rows + 4, n + 8, device="cuda").to(BF16)
        before = big.clone()
        want = mc2.mc2_quant_matmul(x, xs, w, ws, residual=before[:rows, :n])
        r = mc2.mc2_quant_matmul(x, xs, w, ws, residual=big[:rows, :n], out=big[:rows, :n])
        assert r.data_ptr() == big.data_ptr() and torch.equal(big[:rows, :n], want)
        assert torch.equal(big[rows:], before[rows:]) and torch.equal(big[:, n:], before[:, n:])


def test_more_dimensions():
    x, xs, w, ws = make(24, 128, 256, 13)
    a = mc2.mc2_quant_matmul(x.view(2, 3, 4, 256), xs.view(2, 3, 4), w, ws)
    assert a.shape == (2, 3, 4, 128) and torch.equal(a.view(24, 128), mc2.mc2_quant_matmul(x, xs, w, ws))
