"""The operators around the fused linears, as they are measured: the residual
RMS norm with its 8-bit output and its gradient, and the matrix product with
bias, activation and residual in its epilogue and the activation gradient in
its backward product.

Each case is one call with the inputs a user's program holds at that point.
Where ``own`` is false the operators run in their plain form (elementary torch
operations in 32 bits, rounded once at the end); where it is true the calls go
to the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
# exponent of the largest power of two the 8-bit float holds (mx scales)
EMAX = {"e4m3": 8, "e5m2": 15}
GROUP = {"group": 128, "mx": 32}
EPS = 1e-6

# the largest listed case's operations: no drawn case costs more
MOST_FLOPS = 2 * 8192 * 8192 * 7168
MOST_ELEMENTS = 8192 * 8192


def listed():
    return [
        # one decoded token: norm of the hidden state before the next block (latency)
        dict(name="norm-token", op="norm", m=1, h=4096, dtype="bf16", residual=True, quant="none", q="none"),
        # a prompt's tokens into the int8 product with per-token scales
        dict(name="norm-prompt-int8", op="norm", m=4096, h=8192, dtype="bf16", residual=True, quant="token", q="int8"),
        # an odd number of tokens into an fp8 product with per-token scales
        dict(name="norm-ragged-e4m3", op="norm", m=1037, h=7168, dtype="fp16", residual=True, quant="token", q="e4m3"),
        # training's largest step: the norm's backward over all tokens
        dict(name="norm-grad-train", op="norm_grad", m=8192, h=8192, dtype="bf16", residual=True),
        # a short, odd batch of a narrow model's backward
        dict(name="norm-grad-ragged", op="norm_grad", m=333, h=1000, dtype="fp16", residual=False),
        # one decoded token through an up projection (reads the weight once)
        dict(name="linear-token", op="linear", m=1, n=8192, k=4096, dtype="bf16", act="silu", bias=False,
             residual=False, preact=False, w_is_nk=True),
        # a batch of decoded sequences through a down projection, added to the residual
        dict(name="linear-batch", op="linear", m=24, n=4096, k=8192, dtype="fp16", act="none", bias=True,
             residual=True, preact=False, w_is_nk=True),
        # a ragged chunk of a prompt, a slice of a wider activation, through a projection of odd width
        dict(name="linear-ragged", op="linear", m=777, n=1000, k=2056, dtype="bf16", act="relu", bias=True,
             residual=True, preact=False, w_is_nk=False, wide=True),
        # training's forward up projection: the pre-activation is kept for the backward
        dict(name="linear-train", op="linear", m=8192, n=8192, k=7168, dtype="bf16", act="gelu", bias=True,
             residual=False, preact=True, w_is_nk=True),
        # its backward: the down projection's input gradient times the activation's derivative
        dict(name="act-grad-train", op="act_grad", m=8192, n=8192, k=4096, dtype="bf16", act="gelu", w_is_nk=True),
        # the same for a short fine-tuning batch
        dict(name="act-grad-short", op="act_grad", m=197, n=4096, k=4096, dtype="fp16", act="silu", w_is_nk=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "linear", "linear", "act_grad"])
    if op in ("norm", "norm_grad"):
        h = _log_int(rng, 256, 16384, rng.choice([1, 8, 8, 128]))
        m = _log_int(rng, 1, min(16384, MOST_ELEMENTS // h))
        c = dict(op=op, m=m, h=h, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), residual=rng.random() < 0.7)
        if op == "norm":
            c["quant"] = rng.choice(["none", "token", "token", "group", "mx"])
            c["q"] = {"none": ["none"], "mx": ["e4m3", "e5m2"]}.get(c["quant"], ["int8", "int8", "e4m3"])
            c["q"] = rng.choice(c["q"])
            c["wide"] = rng.random() < 0.2
        return c
    n = _log_int(rng, 64, 16384, 8)
    k = _log_int(rng, 64, 16384, 8)
    m = _log_int(rng, 1, max(1, min(16384, MOST_FLOPS // (2 * n * k))))
    c = dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "bf16", "fp16"]), w_is_nk=rng.random() < 0.7,
             act=rng.choice(["relu", "gelu", "gelu_tanh", "silu"]))
    if op == "linear":
        c["act"] = rng.choice(["none", c["act"]])
        c["bias"] = rng.random() < 0.5
        c["residual"] = rng.random() < 0.5
        c["preact"] = rng.random() < 0.3
        c["wide"] = rng.random() < 0.2
    return c


# ------------------------------------------------------------------ inputs

def _within(x, case):
    """x, or x as the first columns of a wider activation (one part of a fused projection's output)."""
    if not case.get("wide"):
        return x
    m, h = x.shape
    wide = torch.zeros(m, -(-h // 8) * 8 + 64, dtype=x.dtype, device=x.device)
    wide[:, :h] = x
    return wide[:, :h]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)

    s = dict(case=case, dt=dt)
    if case["op"] in ("norm", "norm_grad"):
        m, h = case["m"], case["h"]
        # hidden states: tokens of different size and a few channels six times larger
        size = torch.exp(normal(m, 1, std=0.5))
        channel = torch.where(torch.rand(h, generator=g, device="cuda") < 0.01, 6.0, 1.0)
        s["x"] = _within(normal(m, h).mul_(size).mul_(channel).to(dt), case)
        s["weight"] = (1.0 + normal(h, std=0.1)).to(dt)
        if case["op"] == "norm":
            s["residual"] = normal(m, h).mul_(size).to(dt) if case["residual"] else None
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = normal(m, h, std=0.1).to(dt)
            s["dres"] = normal(m, h, std=0.1).to(dt) if case["residual"] else None
        return s
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "linear":
        s["x"] = _within(normal(m, k).to(dt), case)
        s["w"] = normal(*((n, k) if case["w_is_nk"] else (k, n)), std=k ** -0.5).to(dt)
        s["bias"] = normal(n, std=0.1).to(dt) if case["bias"] else None
        s["residual"] = normal(m, n).to(dt) if case["residual"] else None
    else:
        # the layer that follows maps k features to n outputs
        s["dy"] = normal(m, n, std=0.1).to(dt)
        s["w"] = normal(*((n, k) if case["w_is_nk"] else (k, n)), std=k ** -0.5).to(dt)
        s["z"] = normal(m, k).to(dt)
    return s


# ------------------------------------------------------------------ the calls

def run(state):
    return _run_own(state) if own else _run_plain(state)


_mc2 = None


def _package():
    global _mc2
    if _mc2 is None:
        import quantized_gemm_rank_gb300
        _mc2 = quantized_gemm_rank_gb300
    return _mc2


def _run_own(s):
    mc2, c = _package(), s["case"]
    if c["op"] == "norm":
        modes = {"none": mc2.QUANT_NONE, "token": mc2.QUANT_PERTOKEN_DYNAMIC, "group": mc2.QUANT_PERGROUP,
                 "mx": mc2.QUANT_MX}
        q_dtype = torch.int8 if c["q"] in ("int8", "none") else FP8[c["q"]]
        r = mc2.mc2_add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant_mode=modes[c["quant"]],
                                 q_dtype=q_dtype)
        out = {}
        if c["quant"] == "none":
            out["out"] = r["out"]
        else:
            out["q"], out["scale"] = _values(c, r["q"], r["scale"])
        if c["residual"]:
            out["residual"] = r["residual"]
        return out
    if c["op"] == "norm_grad":
        dx, dw = mc2.mc2_rms_norm_grad(s["dy"], s["x"], s["weight"], s["rstd"], dres=s["dres"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "linear":
        out, z = mc2.mc2_matmul_bias_act(s["x"], s["w"], w_is_nk=c["w_is_nk"], bias=s["bias"], activation=c["act"],
                                         residual=s["residual"], with_preact=c["preact"])
        return {"out": out, "preact": z} if c["preact"] else {"out": out}
    return {"dz": mc2.mc2_matmul_act_grad(s["dy"], s["w"], s["z"], activation=c["act"], w_is_nk=c["w_is_nk"])}


def _values(c, q, scale):
    """What the 8-bit codes stand for.  fp8 codes with one scale per token are values already and come with their
    scales; int8 codes and codes with a scale per group are multiplied out (in one pass, to 16 bits)."""
    if c["quant"] == "token" and c["q"] != "int8":
        return q, scale
    if c["quant"] == "token":
        v = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        return torch.mul(q, scale.unsqueeze(1), out=v), scale
    if scale.dtype == torch.uint8:
        scale = torch.ldexp(torch.ones((), device=q.device), scale.int() - 127)
    v = q.to(torch.bfloat16)   # exact: every 8-bit code is a bf16 value
    m, h = q.shape
    size = GROUP[c["quant"]]
    whole = h - h % size
    if whole:
        at = v[:, :whole].unflatten(1, (-1, size))
        torch.mul(at, scale[:, :whole // size].unsqueeze(2), out=at)
    if whole < h:
        torch.mul(v[:, whole:], scale[:, whole // size:], out=v[:, whole:])
    return v, None


# ------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_derivative(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-z))
        return e * (1.0 + z * (1.0 - e))
    return torch.ones_like(z)


def _grouped_absmax(y, group):
    m, h = y.shape
    pad = -h % group
    a = torch.cat([y.abs(), y.new_zeros(m, pad)], dim=1) if pad else y.abs()
    return a.view(m, -1, group).amax(2)


def _run_plain(s):
    c, dt = s["case"], s["dt"]
    if c["op"] == "norm":
        v = s["x"].float()
        if c["residual"]:
            v = v + s["residual"].float()
        y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        out = {}
        if c["quant"] == "none":
            out["out"] = y.to(dt)
        else:
            q, scale = _quantise(y, c["quant"], c["q"])
            out["q"], out["scale"] = _values(c, q, scale)
        if c["residual"]:
            out["residual"] = v.to(dt)
        return out
    if c["op"] == "norm_grad":
        r = s["rstd"].unsqueeze(1)
        xhat = s["x"].float() * r
        g = s["dy"].float() * s["weight"].float()
        dx = r * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(dt), "dw": (s["dy"].float() * xhat).sum(0).to(dt)}
    if c["op"] == "linear":
        w = s["w"].float()
        z = s["x"].float() @ (w.t() if c["w_is_nk"] else w)
        if c["bias"]:
            z = z + s["bias"].float()
        o = _act(z, c["act"])
        if c["residual"]:
            o = o + s["residual"].float()
        return {"out": o.to(dt), "preact": z.to(dt)} if c["preact"] else {"out": o.to(dt)}
    w = s["w"].float()
    dx = s["dy"].float() @ (w if c["w_is_nk"] else w.t())
    return {"dz": (dx * _act_derivative(s["z"].float(), c["act"])).to(dt)}


def _quantise(y, quant, kind):
    if quant == "mx":
        a = _grouped_absmax(y, 32)
        e = torch.where(a > 0, torch.frexp(a).exponent - 1 - EMAX[kind], -127).clamp(-127, 127)
        step, scale = torch.ldexp(torch.ones_like(a), e), (e + 127).to(torch.uint8)
    else:
        a = y.abs().amax(1, keepdim=True) if quant == "token" else _grouped_absmax(y, 128)
        step = a / QMAX[kind]
        scale = step.squeeze(1) if quant == "token" else step
    if quant != "token":
        step = step.repeat_interleave(GROUP[quant], dim=1)[:, :y.shape[1]]
    r = torch.where(step > 0, y / step, 0.0).clamp(-QMAX[kind], QMAX[kind])
    return (torch.round(r).to(torch.int8) if kind == "int8" else r.to(FP8[kind])), scale


# ------------------------------------------------------------------ work and the definition in 64 bits

def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "norm":
        m, h = c["m"], c["h"]
        b = m * h * e * (3 if c["residual"] else 1) + h * e
        if c["quant"] == "none":
            b += m * h * e
        else:
            b += m * h + (4 * m if c["quant"] == "token" else
                          4 * m * -(-h // 128) if c["quant"] == "group" else m * -(-h // 32))
        return {"bytes": b, "flops": 6 * m * h}
    if c["op"] == "norm_grad":
        m, h = c["m"], c["h"]
        return {"bytes": m * h * e * (4 if c["residual"] else 3) + 2 * h * e + 4 * m, "flops": 10 * m * h}
    m, n, k = c["m"], c["n"], c["k"]
    if c["op"] == "linear":
        outs = 1 + (1 if c["residual"] else 0) + (1 if c["preact"] else 0)
        return {"bytes": 2 * (m * k + n * k + m * n * outs + (n if c["bias"] else 0)), "flops": 2 * m * n * k}
    return {"bytes": 2 * (m * n + n * k + 2 * m * k), "flops": 2 * m * n * k}


def _round8(r, kind):
    """Values of 64 bits to the nearest value the 8-bit type holds, ties to even, in 64 bits."""
    if kind == "int8":
        return torch.round(r).clamp(-127, 127)
    bits, least = (3, -6) if kind == "e4m3" else (2, -14)
    ulp = torch.ldexp(torch.ones_like(r), torch.frexp(r).exponent.clamp(min=least + 1) - 1 - bits)
    return (torch.round(r / ulp) * ulp).clamp(-QMAX[kind], QMAX[kind])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = {name: v.double() for name, v in s.items() if isinstance(v, torch.Tensor)}
    if c["op"] == "norm":
        v = d["x"] + d["residual"] if c["residual"] else d["x"]
        y = v / torch.sqrt((v * v).sum(1, keepdim=True) / c["h"] + EPS) * d["weight"]
        out = {}
        if c["quant"] == "none":
            out["out"] = y
        else:
            m, h = y.shape
            size = {"token": h, "group": 128, "mx": 32}[c["quant"]]
            full = torch.zeros(m, -(-h // size) * size, dtype=torch.float64, device=y.device)
            full[:, :h] = y
            full = full.view(m, -1, size)
            top = full.abs().max(2, keepdim=True).values
            if c["quant"] == "mx":
                step = torch.exp2(torch.floor(torch.log2(top)) - EMAX[c["q"]])
            else:
                step = top / QMAX[c["q"]]
            codes = _round8(torch.where(top > 0, full / step, 0.0), c["q"])
            if c["quant"] == "token" and c["q"] != "int8":
                out["q"], out["scale"] = codes.reshape(m, -1)[:, :h], step.reshape(m)
            else:
                out["q"] = (codes * step).reshape(m, -1)[:, :h]
                out["scale"] = step.reshape(m) if c["quant"] == "token" else None
        if c["residual"]:
            out["residual"] = v
        return out
    if c["op"] == "norm_grad":
        # with u = x * rstd and G = dy * w: the gradient of x through its own row's norm
        u = d["x"] * d["rstd"][:, None]
        G = d["dy"] * d["weight"]
        dx = d["rstd"][:, None] * (G - u * ((G * u).sum(1, keepdim=True) / c["h"]))
        return {"dx": dx + d["dres"] if c["residual"] else dx, "dw": torch.einsum("th,th->h", d["dy"], u)}
    if c["op"] == "linear":
        z = torch.einsum("mk,nk->mn" if c["w_is_nk"] else "mk,kn->mn", d["x"], d["w"])
        if c["bias"]:
            z += d["bias"]
        o = _exact_act(z, c["act"])
        if c["residual"]:
            o = o + d["residual"]
        return {"out": o, "preact": z} if c["preact"] else {"out": o}
    dx = torch.einsum("mn,nk->mk" if c["w_is_nk"] else "mn,kn->mk", d["dy"], d["w"])
    z = d["z"].requires_grad_()
    with torch.enable_grad():
        _exact_act(z, c["act"]).sum().backward()   # the derivative by the chain rule, not by its formula
    return {"dz": dx * z.grad}


def _exact_act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2.0)) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z
