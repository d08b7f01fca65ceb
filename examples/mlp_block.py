"""An MLP block on one GPU: the residual norm, the up projection with its
activation, the down projection with the residual, and their backward; the same
block for single tokens in a CUDA graph; and the norm's int8 codes into the
all-to-all product, its per-group codes into the quantised all-reduce.

  python examples/mlp_block.py [--tokens 2048] [--hidden 4096] [--ffn 8192]

Prints each step's time and how far the block is from the same one in 64 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_rank_gb300 as mc2  # noqa: E402


class Block:
    """y = s + W2 act(W1 norm(s) + b1) + b2 with s = x + residual."""

    def __init__(self, hidden, ffn, seed=0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.norm = 1 + normal(hidden, std=0.1)
        self.w1, self.b1 = normal(ffn, hidden, std=hidden ** -0.5), normal(ffn, std=0.1)
        self.w2, self.b2 = normal(hidden, ffn, std=ffn ** -0.5), normal(hidden, std=0.1)

    def forward(self, x, residual, keep=False):
        n = mc2.mc2_add_rms_norm(x, self.norm, residual=residual, with_rstd=keep)
        h, z = mc2.mc2_matmul_bias_act(n["out"], self.w1, bias=self.b1, activation="gelu_tanh", with_preact=keep)
        y, _ = mc2.mc2_matmul_bias_act(h, self.w2, bias=self.b2, residual=n["residual"])
        return y, (n, h, z)

    def backward(self, dy, kept):
        n, h, z = kept
        dz = mc2.mc2_matmul_act_grad(dy, self.w2, z, activation="gelu_tanh")
        dw2, db2 = mc2.mc2_matmul_weight_grad(dy, h)
        dw1, db1 = mc2.mc2_matmul_weight_grad(dz, n["out"])
        dn, _ = mc2.mc2_matmul_bias_act(dz, self.w1, w_is_nk=False)
        dx, dnorm = mc2.mc2_rms_norm_grad(dn, n["residual"], self.norm, n["rstd"], dres=dy)
        return {"x": dx, "norm": dnorm, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}

    def plain(self, x, residual, dy):
        p = {k: v.double().requires_grad_() for k, v in
             (("x", x), ("norm", self.norm), ("w1", self.w1), ("b1", self.b1), ("w2", self.w2), ("b2", self.b2))}
        s = p["x"] + residual.double()
        n = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * p["norm"]
        z = n @ p["w1"].t() + p["b1"]
        h = z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
        y = h @ p["w2"].t() + p["b2"] + s
        y.backward(dy.double())
        return y.detach(), {k: v.grad for k, v in p.items()}


def microseconds(f, reps=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / reps


def off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=8192)
    a = ap.parse_args()
    block = Block(a.hidden, a.ffn)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(m, std=1.0):
        return (torch.randn(m, a.hidden, generator=g, device="cuda") * std).to(torch.bfloat16)

    # training: forward and backward
    x, r, dy = rows(a.tokens), rows(a.tokens), rows(a.tokens, 0.1)
    y, kept = block.forward(x, r, keep=True)
    grads = block.backward(dy, kept)
    few = min(a.tokens, 512)
    ys, ks = block.forward(x[:few], r[:few], keep=True)
    want, wgrads = block.plain(x[:few], r[:few], dy[:few])
    gs = block.backward(dy[:few], ks)
    print(f"forward, {a.tokens} tokens: {microseconds(lambda: block.forward(x, r, keep=True)):.1f} us")
    print(f"backward: {microseconds(lambda: block.backward(dy, kept)):.1f} us ({len(grads)} gradients)")
    print("relative error against 64 bits:", ", ".join([f"y {off(ys, want):.1e}"] + [f"d{k} {off(v, wgrads[k]):.1e}" for k, v in gs.items()]))

    # a decoded token: the block in a CUDA graph, on buffers that are updated in place
    tx, tr = rows(1), rows(1)
    block.forward(tx, tr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ty, _ = block.forward(tx, tr)
    print(f"one token, captured: {microseconds(graph.replay, 200):.1f} us")

    # the norm's int8 codes into the all-to-all product (four ranks' column blocks of the hidden state)
    ranks = 4
    c = mc2.mc2_add_rms_norm(x, block.norm, residual=r, quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC, with_out=True)
    chunks = [c["q"][:, i * (a.hidden // ranks):(i + 1) * (a.hidden // ranks)].contiguous() for i in range(ranks)]
    w8 = torch.randint(-127, 128, (a.hidden, a.ffn), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.full((a.ffn,), a.hidden ** -0.5 / 73, device="cuda")
    out = mc2.mc2_alltoall_quant_mm(chunks, w8, ws, torch.zeros(a.ffn, device="cuda"), x1_quant_mode=mc2.QUANT_PERTOKEN,
                                    x1_scale=c["scale"])["out"]
    print(f"int8 product of the norm's codes against its 16-bit output: {off(out[:64], c['out'][:64].double() @ (w8.double() * ws.double())):.1e}")

    # ... and codes with a scale for each 128 columns through the quantised all-reduce
    two = [mc2.mc2_add_rms_norm(v, block.norm, quant_mode=mc2.QUANT_PERGROUP, with_out=True) for v in (x, r)]
    total = mc2.mc2_quant_all_reduce([t["q"] for t in two], [t["scale"] for t in two], out_dtype=torch.bfloat16)
    print(f"all-reduce of two norms' per-group codes: {off(total, two[0]['out'].double() + two[1]['out'].double()):.1e}")
    assert mc2.mc2_device_status() == mc2.MC2_OK


if __name__ == "__main__":
    main()
