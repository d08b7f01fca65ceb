"""mc2_act_quant, mc2_act_dequant and mc2_act_grad_quant against a plain implementation in 64 bits.

Bounds.  y = act(z) is within OWN (1 + |z|) of the 64-bit value (nothing without an activation).  A scale is the largest |y| times the
rounded 1 / Q, rounded: 2^-23 relative, and y's own error.  A code is the nearest to y / scale: half a
step of the type at that value, plus y's error in units of the scale and 2^-23 relative for the quotient.  A
value is code times scale, rounded in fp32, and its activation; an output is rounded once to its type.
"""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
I8, E4M3, E5M2 = torch.int8, torch.float8_e4m3fn, torch.float8_e5m2
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF16: 1e-38, F16: 2.0 ** -25, F32: 1e-44}
QMAX = {I8: 127.0, E4M3: 448.0, E5M2: 57344.0}
TOKEN, GROUP, MX = mc2.QUANT_PERTOKEN_DYNAMIC, mc2.QUANT_PERGROUP, mc2.QUANT_MX
OWN = 2.0 ** -18
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
KINDS = [(TOKEN, I8), (TOKEN, E4M3), (TOKEN, E5M2), (GROUP, I8), (GROUP, E4M3), (GROUP, E5M2), (MX, E4M3), (MX, E5M2)]


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
    if act == "relu":   # (0 at 0)
        return (z > 0).double()
    z = z.double().clone().requires_grad_()
    plain_act(z, act).sum().backward()
    return z.grad


def exponent(t):
    """Of the largest power of two that is not above t (a logarithm's floor may miss a power of two)."""
    return torch.frexp(t).exponent - 1


def power(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)


def size_of(mode, h):
    return {TOKEN: h, GROUP: 128, MX: 32}[mode]


def grouped(t, mode):
    """(m, groups, size), zeros behind the last column."""
    m, h = t.shape
    size = size_of(mode, h)
    full = torch.zeros(m, -(-h // size) * size, dtype=torch.float64, device=t.device)
    full[:, :h] = t
    return full.view(m, -1, size)


def step_of(scale):
    """Scales (m), (m, groups) as fp64 (m, groups)."""
    s = scale.double() if scale.dtype == F32 else torch.where(scale == 255, torch.nan, power(scale.int() - 127))
    return s.view(s.shape[0], -1)


def spread(scale, mode, h):
    return step_of(scale).repeat_interleave(size_of(mode, h), 1)[:, :h]


def half_step(r, kind):
    if kind == I8:
        return torch.full_like(r, 0.5)
    bits, least = (3, -6) if kind == E4M3 else (2, -14)
    return power(exponent(r.abs().clamp(min=2.0 ** least)) - bits - 1)


def cut(t, wide):
    if not wide:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + wide), 3.0, dtype=t.dtype)
    big[:, 1:1 + t.shape[1]] = t
    return big.cuda()[:, 1:1 + t.shape[1]]


def tensor(m, h, dtype, seed, wide=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(m, h, generator=g) * torch.exp(torch.randn(m, 1, generator=g) * 0.5)
    z[:, :: 37] *= 6
    return cut(z.to(dtype), wide)


def check_quant(z, act, mode, kind):
    q, scale = mc2.mc2_act_quant(z, activation=act, quant_mode=mode, q_dtype=kind)
    m, h = z.shape
    assert q.shape == (m, h) and q.dtype == kind
    y = plain_act(z.double(), act)
    off = OWN * (1 + z.double().abs()) if act != "none" else torch.zeros_like(y)
    top, slack = grouped(y, mode).abs().amax(2), grouped(off, mode).amax(2)
    got = step_of(scale)
    if mode == MX:
        lo, hi = ((top + s * slack).clamp(min=0) for s in (-1, 1))
        emax = 8 if kind == E4M3 else 15
        low, high = (power((torch.where(t > 0, exponent(t), -1000) - emax).clamp(-127, 127)) for t in (lo, hi))
        assert ((got == low) | (got == high)).all()
    else:
        assert ((got - top / QMAX[kind]).abs() <= 2.0 ** -23 * top / QMAX[kind] + slack / QMAX[kind] + 1e-45).all()
    step = spread(scale, mode, h)
    r = torch.where(step > 0, y / step, 0.0).clamp(-QMAX[kind], QMAX[kind])
    off = torch.where(step > 0, off / step, 0.0)
    bad = ~((q.double() - r).abs() <= half_step(r.abs() + off, kind) + off + 2.0 ** -23 * r.abs())
    assert not bad.any(), f"{act} {mode} {kind}: {int(bad.sum())} codes of {bad.numel()} outside"
    return q, scale


SIZES = [(1, 1), (1, 4096), (1, 8192), (2, 31), (3, 32), (5, 33), (1, 127), (4, 128), (3, 129), (7, 1000), (9, 1024), (33, 264),
         (2, 8200), (130, 2048), (3, 16384), (2, 16392), (2, 33000), (1, 70001), (1037, 520), (5000, 40)]


@pytest.mark.parametrize("m,h", SIZES)
@pytest.mark.parametrize("mode,kind", KINDS)
def test_codes(m, h, mode, kind):
    i = SIZES.index((m, h)) + KINDS.index((mode, kind))
    check_quant(tensor(m, h, [BF16, F16, F32][i % 3], i), ACTS[i % 5], mode, kind)


@pytest.mark.parametrize("m,h", [(6, 200), (3, 4096), (2, 1001), (40, 264)])
@pytest.mark.parametrize("mode,kind", KINDS)
@pytest.mark.parametrize("wide", [0, 1, 8, 24])
def test_codes_of_strided_rows(m, h, mode, kind, wide):
    for dtype in (BF16, F32):
        z = tensor(m, h, dtype, 5, wide)
        q, scale = check_quant(z, "none", mode, kind)
        q2, s2 = mc2.mc2_act_quant(z.contiguous(), quant_mode=mode, q_dtype=kind)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale, s2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("h", [512, 1000, 77, 6000])
@pytest.mark.parametrize("mode,kind", [k for k in KINDS if k[0] != MX])
def test_codes_are_torchs(h, dtype, mode, kind):
    """Without an activation, bit for bit what torch's own operations give (each is one fp32 operation)."""
    z = tensor(300, h, dtype, 2)
    q, scale = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind)
    want = grouped(z, mode).abs().amax(2).float() * torch.tensor(1.0 / QMAX[kind], dtype=F32, device="cuda")
    assert torch.equal(scale.view(300, -1), want)
    r = (z.float() / spread(scale, mode, h).float()).clamp(-QMAX[kind], QMAX[kind])
    assert torch.equal(q.double(), (r.round() if kind == I8 else r.to(kind)).double())


@pytest.mark.parametrize("h", [512, 1000])
@pytest.mark.parametrize("mode,kind", KINDS)
def test_codes_are_the_norms(h, mode, kind):
    """A norm's fp32 output is what its codes are made from: kept by itself its scales are the same, to the last bit or
    (mx) equal, and a code at most the next one."""
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(17, h, generator=g).cuda(), torch.rand(h, generator=g).cuda()
    n = mc2.mc2_add_rms_norm(x, w, quant_mode=mode, q_dtype=kind, with_out=True)
    q, s = mc2.mc2_act_quant(n["out"], quant_mode=mode, q_dtype=kind)
    if mode == MX:
        assert torch.equal(n["q"].view(torch.uint8), q.view(torch.uint8)) and torch.equal(n["scale"], s)
    else:
        assert ((n["scale"] - s).abs() <= 2.0 ** -23 * s).all()
        assert ((n["q"].double() - q.double()).abs() <= 2 * half_step(torch.maximum(n["q"].double().abs(), q.double().abs()), kind)).all()


@pytest.mark.parametrize("h", [256, 4099])
@pytest.mark.parametrize("mode,kind", KINDS)
def test_not_numbers_zeros_and_the_ends_of_the_range(h, mode, kind):
    z = tensor(8, h, F32, 7)
    z[0] = 0
    z[1, 40], z[2, 41] = float("nan"), float("inf")
    z[3] = 1e-41          # scales that underflow, or nearly
    z[4] *= 1e37 / z[4].abs().max()
    z[5, :32] = 0
    q, scale = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind)
    v = mc2.mc2_act_dequant(q, scale, dtype=F32)
    step = spread(scale, mode, h)
    group = torch.arange(h, device="cuda") // size_of(mode, h) == 40 // size_of(mode, h)
    assert (q.double()[0] == 0).all() and (v[0] == 0).all()
    assert v[1:3, group].isnan().all() and (q.double()[1:3, group] == 0).all()
    assert v[1:3, ~group].isfinite().all()
    assert (step[1, group].isnan() if mode != MX else scale[1, 1 if size_of(mode, h) == 32 else 0] == 255).all()
    for row in (4, 5, 6, 7):
        bound = spread(scale[row:row + 1], mode, h) * half_step(z[row:row + 1].double() / spread(scale[row:row + 1], mode, h).clamp(min=1e-300), kind)
        if mode != MX:   # (mx codes saturate in the top binade)
            assert ((v[row].double() - z[row].double()).abs() <= bound * (1 + 1e-5) + 2.0 ** -22 * z[row].double().abs()).all()
    assert v[3].isfinite().all() and (v[3].abs() <= 3e-41).all()


def codes(m, h, mode, kind, seed):
    """Codes and scales by plain operations, every code of the type among them where there is room."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (m, h), generator=g).to(torch.uint8).view(kind)
    if kind != I8:
        q = torch.where(q.float().isfinite(), q.float(), 1.0).to(kind)
    if mode == MX:
        scale = torch.randint(117, 122 if kind == E4M3 else 118, (m, -(-h // 32)), generator=g).to(torch.uint8)
        if kind == E5M2:
            scale = scale - 14
    else:
        scale = (torch.rand(m, generator=g) if mode == TOKEN else torch.rand(m, -(-h // 128), generator=g)) * 8 / QMAX[kind]
    return q.cuda(), scale.cuda()


@pytest.mark.parametrize("m,h", [s for s in SIZES if s[0] * s[1] <= 300000])
@pytest.mark.parametrize("mode,kind", KINDS)
def test_values_and_gradients(m, h, mode, kind):
    i = SIZES.index((m, h)) + KINDS.index((mode, kind))
    q, scale = codes(m, h, mode, kind, i)
    z = q.double() * spread(scale, mode, h)
    act = ACTS[i % 5]
    for dtype in (BF16, F16, F32):
        out = mc2.mc2_act_dequant(q, scale, activation=act, dtype=dtype)
        if act == "none":
            # one product in fp32, one rounding
            assert torch.equal(out, (q.float() * spread(scale, mode, h).float()).to(dtype))
        ref = plain_act(z, act)
        bound = (UNIT[dtype] + 2 * 2.0 ** -24) * ref.abs() + (1.2 * 2.0 ** -24 * z.abs() + OWN * (1 + z.abs()) if act != "none" else 0) + LEAST[dtype]
        assert ((out.double() - ref).abs() <= bound).all(), (act, dtype)
    for dtype, wide in ((BF16, 0), (F16, 9), (BF16, 8)):
        dy = tensor(m, h, dtype, i, wide)
        dz = mc2.mc2_act_grad_quant(dy, q, scale, activation=act)
        ref = dy.double() * plain_derivative(z, act)
        # the derivative's own error, and its slope (below 1) times z's rounding
        bound = dy.double().abs() * (2.0 ** -17 * (1 + z.abs()) if act not in ("none", "relu") else 0) + (UNIT[dtype] + 2.0 ** -23) * ref.abs() + LEAST[dtype]
        assert ((dz.double() - ref).abs() <= bound).all(), (act, dtype)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(act):
    """Of act(z) through mc2_act_dequant in 32 bits, at scales a little larger and smaller: d/ds act(q s) = q act'(q s)."""
    q, scale = codes(40, 256, TOKEN, I8, 3)
    q = torch.where(q == 0, 5, q).to(I8)
    e = 2.0 ** -7
    up, down = (mc2.mc2_act_dequant(q, scale * (1 + s * e), activation=act, dtype=F32).double() for s in (1, -1))
    z = q.double() * scale.double()[:, None]
    slope = (up - down) / (2 * e * z)
    dz = mc2.mc2_act_grad_quant(torch.ones(40, 256, dtype=BF16, device="cuda"), q, scale, activation=act).double()
    # the third derivative is below 2, z up to 8: (e z)^2 / 3; the values' errors over the distance; dz's rounding
    assert ((dz - slope).abs() <= (e * z) ** 2 / 3 + 2 * OWN * (1 + z.abs()) / (e * z.abs()) / 2 + 2.0 ** -8 * 1.2).all()


def test_gradient_in_place():
    for h in (264, 1001):
        q, scale = codes(20, h, GROUP, I8, 1)
        dy = tensor(20, h, BF16, 2)
        want = mc2.mc2_act_grad_quant(dy, q, scale, activation="silu")
        got = mc2.mc2_act_grad_quant(dy, q, scale, activation="silu", dz=dy)
        assert got is dy and torch.equal(got, want)


def test_rows_and_columns_beside_the_output_stay():
    for h in (200, 256, 77):
        q, scale = codes(6, h, TOKEN, E4M3, 4)
        big = torch.full((8, h + 16), 5.0, dtype=BF16, device="cuda")
        mc2.mc2_act_dequant(q, scale, out=big[:6, 8:8 + h])
        assert torch.equal(big[:6, 8:8 + h], mc2.mc2_act_dequant(q, scale))
        assert (big[6:] == 5).all() and (big[:, :8] == 5).all() and (big[:, 8 + h:] == 5).all()


@pytest.mark.parametrize("mode", [TOKEN, GROUP])
def test_offsets_past_32_bits(mode):
    """2.3 thousand million elements: the last rows are what they are by themselves."""
    m, h, last = 70000, 32768, 3
    z = torch.zeros(m, h, dtype=BF16, device="cuda")
    z[-last:] = tensor(last, h, BF16, 1)
    z[12345] = z[-1]
    q, scale = mc2.mc2_act_quant(z, quant_mode=mode)
    q2, s2 = mc2.mc2_act_quant(z[-last:].clone(), quant_mode=mode)
    assert torch.equal(q[-last:], q2) and torch.equal(scale[-last:], s2) and torch.equal(q[12345], q2[-1])
    mc2.mc2_act_grad_quant(z, q, scale, activation="gelu", dz=z)
    assert torch.equal(z[-last:], mc2.mc2_act_grad_quant(tensor(last, h, BF16, 1), q2, s2, activation="gelu"))
    v = mc2.mc2_act_dequant(q, scale, activation="gelu", out=z)
    assert torch.equal(v[-last:], mc2.mc2_act_dequant(q2, s2, activation="gelu")) and not v[-last - 1].any()


def test_more_dimensions():
    z = tensor(24, 256, F16, 1)
    for mode, kind in KINDS:
        q, s = mc2.mc2_act_quant(z.view(2, 12, 256), quant_mode=mode, q_dtype=kind)
        q2, s2 = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind)
        assert q.shape == (2, 12, 256) and torch.equal(q.view(torch.uint8).view(24, -1), q2.view(torch.uint8))
        assert torch.equal(s.reshape(-1), s2.reshape(-1))
        assert torch.equal(mc2.mc2_act_dequant(q, s).view(24, 256), mc2.mc2_act_dequant(q2, s2))
        assert torch.equal(mc2.mc2_act_grad_quant(z.view(2, 12, 256), q, s, activation="relu").view(24, 256),
                           mc2.mc2_act_grad_quant(z, q2, s2, activation="relu"))


@pytest.mark.parametrize("h", [256, 259])
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_infinite_codes_and_nans(h, act):
    # every e5m2 code, infinities and NaN among them: each has its limit, and its neighbours are as without it
    q = (torch.arange(h) % 256).repeat(2, 1).to(torch.uint8)
    q[1] = q[1].roll(5)
    q = q.view(E5M2).cuda()
    scale = torch.ones(2, device="cuda")
    z = q.double()
    low, high, lost, fine = z == -torch.inf, z == torch.inf, z.isnan(), z.isfinite()
    assert low.any() and high.any() and lost.any()
    out = mc2.mc2_act_dequant(q, scale, activation=act, dtype=F32)
    dz = mc2.mc2_act_grad_quant(torch.ones(2, h, dtype=F16, device="cuda"), q, scale, activation=act)
    assert torch.equal(out.isnan(), lost) and (out[high] == torch.inf).all()
    assert (out[low] == -torch.inf).all() if act == "none" else (out[low].abs() <= 1e-14).all()
    known = torch.where(fine, z, 0.0)
    bound = OWN * (1 + known.abs()) + 2.0 ** -22 * known.abs()
    assert ((out.double() - plain_act(known, act)).abs() <= bound)[fine].all()
    if act == "none":
        assert (dz == 1).all()
        return
    assert (dz[lost] == 0).all() if act == "relu" else torch.equal(dz.isnan(), lost)
    assert (dz[high] == 1).all() and (dz[low] == 0).all()
    assert ((dz.double() - plain_derivative(known, act)).abs() <= 2.0 ** -11 * 1.2 + 2.0 ** -17 * (1 + known.abs()))[fine].all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("h", [96, 256, 264, 2048])
@pytest.mark.parametrize("mode,kind", KINDS)
def test_not_numbers_of_16_bits(mode, kind, h, dtype):
    # one in a row each: its group is lost, and the rows and groups beside it are as without it
    z = tensor(9, h, dtype, 9)
    clean_q, clean_scale = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind)
    odd = [float("nan"), float("inf"), -float("inf"), 0.0]
    for i, v in enumerate(odd):
        z[2 * i + 1, 37 + 9 * i] = v
    z.view(torch.int16)[1, 38] = -1   # a NaN with its sign and every bit set
    z[8] = 0
    q, scale = mc2.mc2_act_quant(z, quant_mode=mode, q_dtype=kind)
    step, clean_step = spread(scale, mode, h), spread(clean_scale, mode, h)
    lost = torch.zeros(9, h, dtype=torch.bool, device="cuda")
    same = torch.ones_like(lost)
    for i, v in enumerate(odd):
        group = torch.arange(h, device="cuda") // size_of(mode, h) == (37 + 9 * i) // size_of(mode, h)
        same[2 * i + 1, group] = False
        lost[2 * i + 1, group] = v != 0
    same[8] = False
    assert torch.equal(q.double()[same], clean_q.double()[same]) and torch.equal(step[same], clean_step[same])
    assert not step[lost].isfinite().any() and (q.double()[lost] == 0).all() and step[~lost].isfinite().all()
    assert (q.double()[8] == 0).all() and (step[8] <= 2.0 ** -127).all()
