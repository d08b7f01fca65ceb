"""mc2_add_rms_norm and mc2_rms_norm_grad against a plain implementation in 64 bits.

Bounds.  The kernels' arithmetic is fp32.  A sum over h elements is at most
h/32 sequential additions a thread and then a tree, so its relative error is
below (h/32 + 16) 2^-24 for terms of one sign; rstd takes half of it, and a few
roundings (the reciprocal square root's 2 ulp among them) come on top: E(h) =
(h/32 + 32) 2^-24 relative on y.  An output rounded to bf16, fp16 or fp32 adds
2^-8, 2^-11 or 2^-24 relative (fp16 below 2^-14: 2^-25 absolute).
"""
import math

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, E5M2, I8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.int8
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF16: 1e-38, F16: 2.0 ** -25, F32: 1e-38}
QMAX = {I8: 127.0, E4M3: 448.0, E5M2: 57344.0}


def E(h):
    return (h / 32 + 32) * 2.0 ** -24


def make(m, h, dtype, seed=0, residual=True, w_f32=False, wide=0):
    g = torch.Generator().manual_seed(seed)

    def cut(t):
        if not wide:
            return t.cuda()
        big = torch.full((m, h + wide), 7.0, dtype=t.dtype)
        big[:, :h] = t
        return big.cuda()[:, :h]

    size = torch.exp(torch.randn(m, 1, generator=g))
    x = cut((torch.randn(m, h, generator=g) * size).to(dtype))
    r = cut((torch.randn(m, h, generator=g) * size).to(dtype)) if residual else None
    w = (1 + 0.2 * torch.randn(h, generator=g)).to(F32 if w_f32 else dtype).cuda()
    return x, r, w


def plain(x, r, w, eps):
    """y, s and rstd in 64 bits."""
    s = x.double() + r.double() if r is not None else x.double()
    rstd = 1 / torch.sqrt(s.square().mean(-1) + eps)
    return s * rstd[..., None] * w.double(), s, rstd


def near(got, ref, rel, what, floor=0.0):
    assert got.shape == ref.shape, what
    d = (got.double() - ref).abs()
    bad = ~(d <= rel * ref.abs() + floor)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float((d / (rel * ref.abs() + floor + 1e-300)).max()):.3g} of the bound"


SHAPES = [(1, 1), (1, 8), (1, 4096), (2, 7), (3, 31), (5, 33), (4, 127), (7, 129), (3, 255), (9, 256), (33, 1000),
          (17, 1024), (8, 2047), (6, 2048), (5, 2056), (64, 4096), (3, 5120), (5, 7168), (11, 8192), (2, 8200),
          (3, 12288), (2, 16384), (3, 16392), (2, 20000), (1, 40000), (700, 640)]


@pytest.mark.parametrize("m,h", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_out_residual_rstd(m, h, dtype):
    x, r, w = make(m, h, dtype, seed=m + h, residual=(m + h) % 2 == 0, w_f32=h % 3 == 0)
    y, s, rstd = plain(x, r, w, 1e-5)
    got = mc2.mc2_add_rms_norm(x, w, residual=r, eps=1e-5, with_rstd=True)
    near(got["out"], y, UNIT[dtype] + E(h), "out", LEAST[dtype])
    near(got["rstd"], rstd, E(h), "rstd")
    if r is not None:
        # one rounding to fp32 and one to the type
        near(got["residual"], s, UNIT[dtype] + 2.0 ** -24, "residual", LEAST[dtype])
    else:
        assert got["residual"] is None
    assert got["q"] is None and got["scale"] is None


@pytest.mark.parametrize("m,h", [(1, 1), (3, 33), (2, 127), (5, 256), (9, 1000), (4, 2047), (6, 4096), (3, 8192),
                                 (2, 8200), (3, 16384), (2, 20000)])
@pytest.mark.parametrize("mode,q_dtype", [(mc2.QUANT_PERTOKEN_DYNAMIC, I8), (mc2.QUANT_PERTOKEN_DYNAMIC, E4M3),
                                          (mc2.QUANT_PERTOKEN_DYNAMIC, E5M2), (mc2.QUANT_PERGROUP, I8),
                                          (mc2.QUANT_PERGROUP, E4M3), (mc2.QUANT_MX, E4M3), (mc2.QUANT_MX, E5M2)])
def test_codes_are_those_of_the_unrounded_output(m, h, mode, q_dtype):
    """With fp32 in and out the codes' source is visible: scales and codes must
    be the formula's on it, bit for bit (one IEEE division, one rounding)."""
    x, r, w = make(m, h, F32, seed=3 * m + h)
    x[0, h // 2] *= 30
    got = mc2.mc2_add_rms_norm(x, w, residual=r, quant_mode=mode, q_dtype=q_dtype, with_out=True)
    y, _, _ = plain(x, r, w, 1e-6)
    near(got["out"], y, 2.0 ** -24 + E(h), "out", 1e-38)
    v = got["out"].cpu()
    size = {mc2.QUANT_PERTOKEN_DYNAMIC: h, mc2.QUANT_PERGROUP: 128, mc2.QUANT_MX: 32}[mode]
    groups = -(-h // size)
    pad = torch.zeros(m, groups * size)
    pad[:, :h] = v
    top = pad.view(m, groups, size).abs().amax(2)
    if mode == mc2.QUANT_MX:
        e = torch.where(top > 0, torch.frexp(top).exponent - 1 - (8 if q_dtype == E4M3 else 15), -127).clamp(min=-127)
        assert torch.equal(got["scale"].cpu(), (e + 127).to(torch.uint8))
        step = torch.ldexp(torch.ones_like(top), e)
    else:
        step = top / QMAX[q_dtype]
        assert torch.equal(got["scale"].cpu().view(m, groups), step)
    ratio = (pad.view(m, groups, size) / step[..., None]).view(m, -1)[:, :h]
    if q_dtype == I8:
        want = torch.round(ratio).clamp(-127, 127).to(I8)
        assert torch.equal(got["q"].cpu(), want)
    else:
        want = ratio.clamp(-QMAX[q_dtype], QMAX[q_dtype]).to(q_dtype)
        assert torch.equal(got["q"].cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("mode,q_dtype", [(mc2.QUANT_PERTOKEN_DYNAMIC, I8), (mc2.QUANT_PERTOKEN_DYNAMIC, E4M3),
                                          (mc2.QUANT_PERGROUP, I8), (mc2.QUANT_MX, E5M2)])
@pytest.mark.parametrize("m,h", [(1, 4096), (37, 1000), (5, 8192), (3, 10240), (4, 999)])
def test_codes_stand_for_the_output(m, h, dtype, mode, q_dtype):
    """16-bit in: code x scale is y to half a step of the code (and E(h) on both)."""
    x, r, w = make(m, h, dtype, seed=m * h)
    got = mc2.mc2_add_rms_norm(x, w, residual=r, quant_mode=mode, q_dtype=q_dtype)
    assert got["out"] is None
    y, _, _ = plain(x, r, w, 1e-6)
    scale = got["scale"]
    if mode == mc2.QUANT_MX:
        scale = torch.exp2(scale.double() - 127)
    scale = scale.double().view(m, -1)
    size = {mc2.QUANT_PERTOKEN_DYNAMIC: h, mc2.QUANT_PERGROUP: 128, mc2.QUANT_MX: 32}[mode]
    step = scale.repeat_interleave(size, 1)[:, :h]
    back = got["q"].double() * step
    if q_dtype == I8:
        half = 0.5 * step
    else:
        bits, least = (4, 2.0 ** -10) if q_dtype == E4M3 else (3, 2.0 ** -17)
        half = torch.maximum(y.abs() * 2.0 ** -bits, least * step)
        if mode == mc2.QUANT_MX:   # saturation: up to 2 - 1.75 of the top binade
            half = torch.maximum(half, y.abs() - QMAX[q_dtype] * step)
    assert ((back - y).abs() <= half * (1 + 1e-4) + 2 * E(h) * y.abs() + 1e-30).all()


def test_strided_rows_and_in_place():
    for h in (1000, 1003, 4096):
        x, r, w = make(19, h, BF16, seed=h, wide=8)
        y, s, _ = plain(x, r, w, 1e-6)
        keep = x.clone(), r.clone()
        wide = torch.zeros(19, h + 24, dtype=BF16, device="cuda")
        got = mc2.mc2_add_rms_norm(x, w, residual=r, out=wide[:, :h])
        near(got["out"], y, UNIT[BF16] + E(h), "out into a slice", 1e-38)
        assert (wide[:, h:] == 0).all(), "wrote past its columns"
        # the residual stream updated in place, the output over x
        got = mc2.mc2_add_rms_norm(x, w, residual=r, out=x, residual_out=r)
        near(x, y, UNIT[BF16] + E(h), "out over x", 1e-38)
        near(r, s, UNIT[BF16] + 2.0 ** -24, "residual in place", 1e-38)
        assert (x._base[:, h:] == 7).all() and (r._base[:, h:] == 7).all()
        del keep


def test_three_dimensions_and_a_side_stream():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 5, 256, generator=g).to(F16).cuda()
    w = torch.ones(256, dtype=F16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mc2.mc2_add_rms_norm(x, w, quant_mode=mc2.QUANT_MX, q_dtype=E4M3, with_out=True, with_rstd=True, stream=s)
    s.synchronize()
    y, _, rstd = plain(x, None, w, 1e-6)
    near(got["out"], y, UNIT[F16] + E(256), "out", LEAST[F16])
    assert got["rstd"].shape == (3, 5) and got["scale"].shape == (3, 5, 8) and got["q"].shape == (3, 5, 256)


@pytest.mark.parametrize("h", [512, 777, 8192, 20000])
def test_rows_of_zeros_nan_and_infinity(h):
    """A zero row gives zeros (scale 0); NaN and infinity stay in their rows and
    show in the scale; neighbouring rows are what they are alone."""
    x, _, w = make(5, h, BF16, seed=2, residual=False)
    x[1] = 0
    x[2, h // 3] = math.nan
    x[3, h - 1] = math.inf
    for q_dtype in (I8, E4M3):
        got = mc2.mc2_add_rms_norm(x, w, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, q_dtype=q_dtype, with_out=True)
        alone = mc2.mc2_add_rms_norm(x[4:].clone(), w, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, q_dtype=q_dtype,
                                     with_out=True)
        assert torch.equal(got["out"][4:], alone["out"])
        assert torch.equal(got["q"][4:].view(torch.uint8), alone["q"].view(torch.uint8))
        assert (got["out"][1] == 0).all() and got["scale"][1] == 0 and (got["q"][1].view(torch.uint8) == 0).all()
        assert got["out"][2].isnan().all() and got["scale"][2].isnan() and (got["q"][2].view(torch.uint8) == 0).all()
        assert got["out"][3, h - 1].isnan() and (got["out"][3, :h - 1] == 0).all() and got["scale"][3].isnan()
    mx = mc2.mc2_add_rms_norm(x, w, quant_mode=mc2.QUANT_MX, q_dtype=E4M3)
    assert (mx["scale"][1] == 0).all() and (mx["q"][1].view(torch.uint8) == 0).all()
    assert (mx["scale"][2] == 255).all() and mx["scale"][3, -1] == 255 and (mx["scale"][3, :-1] == 0).all()


def test_largest_and_smallest_values():
    """fp16 rows at the type's largest value (their squares are past fp16, not past
    fp32) and rows whose squares vanish beside eps."""
    x = torch.full((2, 4096), 65504.0, dtype=F16, device="cuda")
    x[1] = 2.0 ** -24
    w = torch.ones(4096, dtype=F16, device="cuda")
    y, _, _ = plain(x, None, w, 1e-6)
    got = mc2.mc2_add_rms_norm(x, w)
    near(got["out"], y, UNIT[F16] + E(4096), "out", LEAST[F16])


def test_same_bits_every_time():
    x, r, w = make(257, 4104, BF16, seed=8)
    dy, _, _ = make(257, 4104, BF16, seed=9)
    a = mc2.mc2_add_rms_norm(x, w, residual=r, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, with_rstd=True)
    b = mc2.mc2_add_rms_norm(x, w, residual=r, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, with_rstd=True)
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["scale"], b["scale"])
    g1 = mc2.mc2_rms_norm_grad(dy, a["residual"], w, a["rstd"])
    g2 = mc2.mc2_rms_norm_grad(dy, a["residual"], w, a["rstd"])
    assert torch.equal(g1[0], g2[0]) and torch.equal(g1[1], g2[1])


# ------------------------------------------------------------------ gradient

def plain_grad(dy, x, w, rstd, dres):
    xhat = x.double() * rstd.double()[..., None]
    g = dy.double() * w.double()
    c = (g * xhat).mean(-1, keepdim=True)
    dx = rstd.double()[..., None] * (g - xhat * c)
    size = rstd.double()[..., None] * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    if dres is not None:
        dx, size = dx + dres.double(), size + dres.double().abs()
    flat = (dy.double() * xhat).reshape(-1, x.shape[-1])
    return dx, size, flat.sum(0), flat.abs().sum(0)


@pytest.mark.parametrize("m,h", SHAPES + [(305, 64), (609, 1000), (1300, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gradient_against_the_formula(m, h, dtype):
    """dx: E(h) on the size of its terms, one rounding.  dw: a sum of m terms in at
    most m + 304 fp32 additions: (m + 310) 2^-24 on the sum of their sizes."""
    x, dres, w = make(m, h, dtype, seed=m + h, residual=(m + h) % 3 != 0, w_f32=h % 3 == 0)
    dy, _, _ = make(m, h, dtype, seed=m + h + 1, residual=False)
    rstd = mc2.mc2_add_rms_norm(x, w, with_rstd=True)["rstd"]
    dx, dw = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres)
    rdx, size, rdw, wsize = plain_grad(dy, x, w, rstd, dres)
    near(dx, rdx, UNIT[dtype], "dx", E(h) * size + LEAST[dtype])
    near(dw, rdw, UNIT[w.dtype], "dw", (m + 310) * 2.0 ** -24 * wsize + LEAST[w.dtype])
    only, none = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres, with_weight=False)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("m,h", [(3, 64), (5, 1000), (2, 8192)])
def test_gradient_against_differences(m, h):
    """The directional derivative of sum(out * dy) along a random direction, by
    central differences of the 64-bit forward at step 1e-5 (an error near 1e-9
    of its terms), against <dx, direction> and <dw, direction> of the fp32 call."""
    x, _, w = make(m, h, F32, seed=h, residual=False)
    dy, v, u = make(m, h, F32, seed=h + 1)
    got = mc2.mc2_add_rms_norm(x, w, with_rstd=True)
    dx, dw = mc2.mc2_rms_norm_grad(dy, x, w, got["rstd"])
    t = 1e-5

    def f(a, b):
        return (plain(x.double() + a * v.double(), None, w.double() + b * u.double(), 1e-6)[0] * dy.double()).sum()

    for a, b, have in ((t, 0, (dx.double() * v.double())), (0, t, (dw.double() * u.double()))):
        slope = float(f(a, b) - f(-a, -b)) / (2 * t)
        size = float(have.abs().sum())
        assert abs(slope - float(have.sum())) <= (E(h) * 4 + 1e-6) * size


def test_gradient_strided_and_in_place():
    for h in (1000, 1003):
        x, dres, w = make(21, h, F16, seed=h, wide=16)
        dy, _, _ = make(21, h, F16, seed=h + 5, residual=False, wide=16)
        rstd = mc2.mc2_add_rms_norm(x, w, with_rstd=True)["rstd"]
        rdx, size, rdw, wsize = plain_grad(dy, x, w, rstd, dres)
        dx, dw = mc2.mc2_rms_norm_grad(dy, x, w, rstd, dres=dres, dx=dy)
        assert dx.data_ptr() == dy.data_ptr()
        near(dx, rdx, UNIT[F16], "dx over dy", E(h) * size + LEAST[F16])
        near(dw, rdw, UNIT[F16], "dw", (21 + 310) * 2.0 ** -24 * wsize + LEAST[F16])
        assert (dy._base[:, h:] == 7).all()
