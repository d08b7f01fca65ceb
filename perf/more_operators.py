"""The 8-bit path of a linear, as it is measured: the product of int8 codes with scales per token and per channel, an
activation kept in 8 bits (and brought back), and what the backward pass makes of it: the activation's gradient and the
weight's.

Each case is one step with the inputs a user's program holds at that point.  Where ``own`` is false the operators run in
their plain form (elementary torch operations in 32 bits, rounded once at the end); where it is true the calls go to the
package's entry points.
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
ACTS = ["relu", "gelu", "gelu_tanh", "silu"]

# the largest listed case's operations and elements: no drawn case costs more
MOST_FLOPS = 2 * 4096 * 7168 * 8192
MOST_ELEMENTS = 8192 * 8192


def listed():
    return [
        # one decoded token through an int8 projection (latency; reads the weight once)
        dict(name="product-token", op="product", m=1, n=4096, k=4096, dtype="bf16", act="none", bias="none",
             residual=False, w_is_nk=True),
        # a batch of decoded sequences through a down projection, added to the residual
        dict(name="product-batch", op="product", m=48, n=4096, k=8192, dtype="fp16", act="none", bias="fp32",
             residual=True, w_is_nk=True),
        # a ragged chunk of a prompt, a rank's slice of wider codes, through a (k, n) weight of odd width
        dict(name="product-ragged", op="product", m=777, n=1000, k=2056, dtype="bf16", act="silu", bias="same",
             residual=False, w_is_nk=False, wide=True),
        # a whole prompt through an up projection
        dict(name="product-prompt", op="product", m=4096, n=7168, k=8192, dtype="bf16", act="gelu", bias="same",
             residual=False, w_is_nk=True),
        # one decoded token's activation as the int8 input of the next projection (latency)
        dict(name="keep-token", op="keep", m=1, h=8192, dtype="bf16", act="silu", quant="token", q="int8"),
        # an odd number of tokens as the fp8 input of the next product
        dict(name="keep-ragged", op="keep", m=1037, h=7168, dtype="fp16", act="gelu", quant="token", q="e4m3"),
        # training's largest step: pre-activations kept in int8 with a scale per 128 columns, and brought back
        dict(name="keep-train", op="keep", m=8192, h=8192, dtype="bf16", act="none", quant="group", q="int8"),
        # training's backward through the activation of the kept pre-activations
        dict(name="act-grad-train", op="act_grad", m=8192, h=8192, dtype="bf16", act="gelu", quant="group", q="int8"),
        # the same for a short fine-tuning batch of odd width, kept as mx
        dict(name="act-grad-short", op="act_grad", m=197, h=4100, dtype="fp16", act="silu", quant="mx", q="e4m3"),
        # training's weight gradient of a down projection, whose input is made again from the kept pre-activations
        dict(name="weight-train", op="weight", m=8192, n=4096, k=7168, dtype="bf16", act="gelu", quant="group", q="int8"),
        # a short fine-tuning batch of odd sizes, kept as the forward product's codes
        dict(name="weight-short", op="weight", m=333, n=1000, k=4104, dtype="fp16", act="none", quant="token", q="int8"),
        # many tokens through a narrow projection: few outputs, a long sum
        dict(name="weight-long", op="weight", m=16384, n=512, k=1024, dtype="bf16", act="none", quant="mx", q="e4m3"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _kept(rng):
    quant = rng.choice(["token", "token", "group", "mx"])
    return dict(quant=quant, q=rng.choice(["e4m3", "e5m2"] if quant == "mx" else ["int8", "int8", "e4m3"]))


def draw(rng):
    op = rng.choice(["product", "product", "product", "keep", "act_grad", "weight", "weight"])
    if op in ("keep", "act_grad"):
        h = _log_int(rng, 64, 16384, rng.choice([1, 8, 8, 128]))
        m = _log_int(rng, 1, min(16384, MOST_ELEMENTS // h))
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"] if op == "keep" else ["bf16", "bf16", "fp16"])
        # (32-bit tensors that are kept are states and gradients, without an activation)
        acts = ["none"] if dtype == "fp32" else (["none"] * 3 if op == "keep" else []) + ACTS
        return dict(op=op, m=m, h=h, dtype=dtype, act=rng.choice(acts), wide=rng.random() < 0.2, **_kept(rng))
    n = _log_int(rng, 64, 16384, rng.choice([1, 8, 16, 16, 16]))
    k = _log_int(rng, 64, 16384, rng.choice([1, 8, 16, 16, 16]))
    m = _log_int(rng, 1, max(1, min(16384, MOST_FLOPS // (2 * n * k))))
    c = dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "bf16", "fp16"]), wide=rng.random() < 0.2)
    if op == "product":
        return dict(c, act=rng.choice(["none"] * 4 + ACTS), bias=rng.choice(["none", "same", "fp32"]),
                    residual=rng.random() < 0.4, w_is_nk=rng.random() < 0.7)
    return dict(c, act=rng.choice(["none"] * 4 + ACTS), **_kept(rng))


# ------------------------------------------------------------------ inputs

def _within(x, case):
    """x, or x as the first columns of a wider tensor (one part of a fused projection, a rank's slice)."""
    if not case.get("wide"):
        return x
    m, h = x.shape
    wide = torch.zeros(m, -(-h // 16) * 16 + 64, dtype=x.dtype, device=x.device)
    wide[:, :h] = x
    return wide[:, :h]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dt = case, DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)

    def activation(m, h):
        # tokens of different size and a few channels six times larger
        size = torch.exp(normal(m, 1, std=0.5))
        channel = torch.where(torch.rand(h, generator=g, device="cuda") < 0.01, 6.0, 1.0)
        return normal(m, h).mul_(size).mul_(channel)

    s = dict(case=c, dt=dt)
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        x, s["x_scale"] = _quantise(activation(m, k), "token", "int8")
        s["x"] = _within(x, c)
        w, s["w_scale"] = _quantise(normal(n, k, std=k ** -0.5), "token", "int8")
        s["w"] = w if c["w_is_nk"] else w.t().contiguous()
        s["bias"] = {"none": None, "same": dt, "fp32": torch.float32}[c["bias"]]
        if s["bias"] is not None:
            s["bias"] = normal(n, std=0.1).to(s["bias"])
        s["residual"] = normal(m, n).to(dt) if c["residual"] else None
        return s
    if c["op"] == "keep":
        s["z"] = _within(activation(c["m"], c["h"]).to(dt), c)
        return s
    s["q"], s["scale"] = _quantise(activation(c["m"], c["h"] if c["op"] == "act_grad" else c["k"]), c["quant"], c["q"])
    s["dy"] = _within(normal(c["m"], c["h"] if c["op"] == "act_grad" else c["n"], std=0.1).to(dt), c)
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
    if c["op"] == "product":
        return {"out": mc2.mc2_quant_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], w_is_nk=c["w_is_nk"], bias=s["bias"],
                                            activation=c["act"], residual=s["residual"], dtype=s["dt"])}
    if c["op"] == "keep":
        mode = {"token": mc2.QUANT_PERTOKEN_DYNAMIC, "group": mc2.QUANT_PERGROUP, "mx": mc2.QUANT_MX}[c["quant"]]
        q, scale = mc2.mc2_act_quant(s["z"], activation=c["act"], quant_mode=mode,
                                     q_dtype=torch.int8 if c["q"] == "int8" else FP8[c["q"]])
        if c["quant"] == "token" and c["q"] != "int8":
            return {"q": q, "scale": scale}   # fp8 codes are values, in units of their token's scale
        out = {"value": mc2.mc2_act_dequant(q, scale, dtype=s["dt"])}
        return dict(out, scale=scale) if c["quant"] == "token" else out
    if c["op"] == "act_grad":
        return {"dz": mc2.mc2_act_grad_quant(s["dy"], s["q"], s["scale"], activation=c["act"])}
    dw, db = mc2.mc2_matmul_weight_grad_quant(s["dy"], s["q"], s["scale"], activation=c["act"])
    return {"dw": dw, "db": db}


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
    e = 1.0 / (1.0 + torch.exp(-z))
    return e * (1.0 + z * (1.0 - e))


def _grouped_absmax(y, group):
    m, h = y.shape
    pad = -h % group
    a = torch.cat([y.abs(), y.new_zeros(m, pad)], dim=1) if pad else y.abs()
    return a.view(m, -1, group).amax(2)


def _steps(scale, quant, h):
    """Each element's scale in 32 bits, to be multiplied with an (m, h) matrix."""
    if quant == "token":
        return scale.unsqueeze(1)
    if quant == "mx":
        scale = torch.ldexp(torch.ones((), device=scale.device), scale.int() - 127)
    return scale.repeat_interleave(GROUP[quant], dim=1)[:, :h]


def _quantise(y, quant, kind):
    """Codes and scales of a matrix of 32 bits: fp32 scales per row or per 128 columns, e8m0 codes per 32."""
    if quant == "mx":
        a = _grouped_absmax(y, 32)
        e = torch.where(a > 0, torch.frexp(a).exponent - 1 - EMAX[kind], -127).clamp(-127, 127)
        scale = (e + 127).to(torch.uint8)
    else:
        a = y.abs().amax(1) if quant == "token" else _grouped_absmax(y, 128)
        scale = a / QMAX[kind]
    step = _steps(scale, quant, y.shape[1])
    r = torch.where(step > 0, y / step, 0.0).clamp(-QMAX[kind], QMAX[kind])
    return (torch.round(r).to(torch.int8) if kind == "int8" else r.to(FP8[kind])), scale


def _run_plain(s):
    c, dt = s["case"], s["dt"]
    if c["op"] == "product":
        w = s["w"].float()
        z = (s["x"].float() @ (w.t() if c["w_is_nk"] else w)) * s["x_scale"].unsqueeze(1) * s["w_scale"]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        o = _act(z, c["act"])
        if c["residual"]:
            o = o + s["residual"].float()
        return {"out": o.to(dt)}
    if c["op"] == "keep":
        q, scale = _quantise(_act(s["z"].float(), c["act"]), c["quant"], c["q"])
        if c["quant"] == "token" and c["q"] != "int8":
            return {"q": q, "scale": scale}
        out = {"value": (q.float() * _steps(scale, c["quant"], c["h"])).to(dt)}
        return dict(out, scale=scale) if c["quant"] == "token" else out
    z = s["q"].float() * _steps(s["scale"], c["quant"], s["q"].shape[1])
    if c["op"] == "act_grad":
        return {"dz": (s["dy"].float() * _act_derivative(z, c["act"])).to(dt)}
    dy = s["dy"].float()
    return {"dw": (dy.t() @ _act(z, c["act"])).to(dt), "db": dy.sum(0).to(dt)}


# ------------------------------------------------------------------ work and the definition in 64 bits

def _scale_bytes(c, m, h):
    return {"token": 4 * m, "group": 4 * m * -(-h // 128), "mx": m * -(-h // 32)}[c["quant"]]


def work(case):
    c, m = case, case["m"]
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "product":
        n, k = c["n"], c["k"]
        b = m * k + n * k + 4 * (m + n) + 2 * m * n * (2 if c["residual"] else 1)
        return {"bytes": b + n * {"none": 0, "same": 2, "fp32": 4}[c["bias"]], "flops": 2 * m * n * k}
    if c["op"] == "keep":
        # read once, kept; the codes are values themselves or are brought back to the input's type
        h, codes = c["h"], c["m"] * c["h"] + _scale_bytes(c, c["m"], c["h"])
        back = 0 if c["quant"] == "token" and c["q"] != "int8" else codes + m * h * e
        return {"bytes": m * h * e + codes + back, "flops": 10 * m * h}
    if c["op"] == "act_grad":
        return {"bytes": m * c["h"] * (2 * e + 1) + _scale_bytes(c, m, c["h"]), "flops": 12 * m * c["h"]}
    n, k = c["n"], c["k"]
    return {"bytes": e * (m * n + n * k + n) + m * k + _scale_bytes(c, m, k), "flops": 2 * m * n * k}


def _round8(r, kind):
    """Values of 64 bits to the nearest value the 8-bit type holds, ties to even, in 64 bits."""
    if kind == "int8":
        return torch.round(r).clamp(-127, 127)
    bits, least = (3, -6) if kind == "e4m3" else (2, -14)
    ulp = torch.ldexp(torch.ones_like(r), torch.frexp(r).exponent.clamp(min=least + 1) - 1 - bits)
    return (torch.round(r / ulp) * ulp).clamp(-QMAX[kind], QMAX[kind])


def _exact_values(q, scale, quant):
    """What codes stand for, group by group, in 64 bits."""
    m, h = q.shape
    size = {"token": h, "group": 128, "mx": 32}[quant]
    full = torch.zeros(m, -(-h // size) * size, dtype=torch.float64, device=q.device)
    full[:, :h] = q.double()
    step = torch.ldexp(torch.ones_like(scale, dtype=torch.float64), scale.int() - 127) if quant == "mx" else scale.double()
    return (full.view(m, -1, size) * step.reshape(m, -1, 1)).reshape(m, -1)[:, :h]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "product":
        z = torch.einsum("mk,nk->mn" if c["w_is_nk"] else "mk,kn->mn", s["x"].double(), s["w"].double())
        z *= torch.outer(s["x_scale"].double(), s["w_scale"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        o = _exact_act(z, c["act"])
        return {"out": o + s["residual"].double() if c["residual"] else o}
    if c["op"] == "keep":
        y = _exact_act(s["z"].double(), c["act"])
        m, h = y.shape
        size = {"token": h, "group": 128, "mx": 32}[c["quant"]]
        full = torch.zeros(m, -(-h // size) * size, dtype=torch.float64, device=y.device)
        full[:, :h] = y
        full = full.view(m, -1, size)
        top = full.abs().max(2, keepdim=True).values
        if c["quant"] == "mx":   # (a logarithm's floor may miss a power of two)
            step = torch.ldexp(torch.ones_like(top), torch.frexp(top).exponent - 1 - EMAX[c["q"]])
        else:
            step = top / QMAX[c["q"]]
        codes = _round8(torch.where(top > 0, full / step, 0.0), c["q"])
        if c["quant"] == "token" and c["q"] != "int8":
            return {"q": codes.reshape(m, -1)[:, :h], "scale": step.reshape(m)}
        out = {"value": torch.where(top > 0, codes * step, 0.0).reshape(m, -1)[:, :h]}
        return dict(out, scale=step.reshape(m)) if c["quant"] == "token" else out
    z, dy = _exact_values(s["q"], s["scale"], c["quant"]), s["dy"].double()
    if c["op"] == "act_grad":
        z = z.clone().requires_grad_()
        with torch.enable_grad():
            _exact_act(z, c["act"]).sum().backward()   # the derivative by the chain rule, not by its formula
        return {"dz": dy * z.grad}
    return {"dw": torch.einsum("tn,tk->nk", dy, _exact_act(z, c["act"])), "db": torch.einsum("tn->n", dy)}


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
