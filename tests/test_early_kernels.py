"""Kernels that may begin before the stream's previous kernel ends read nothing through the read-only path: what they
read, that kernel may write while they are resident, and read-only loads are for data that nobody writes meanwhile.
(load_settled is for what the call's own first kernel has already waited for.)"""
import glob
import os
import re

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

CSRC = os.path.join(os.path.dirname(os.path.abspath(mc2.__file__)), "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global\.nc|const\s+[\w:]+\s*\*\s*__restrict__")


def definitions(path):
    """(name, text) of the definitions in a source file that are outside of any other but a namespace."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
    text = re.sub(r"^\s*#[^\n]*(?:\\\n[^\n]*)*", "", text, flags=re.M)
    found, depth, start = [], 0, 0
    for at, c in enumerate(text):
        if c == "{":
            if depth == 0 and re.search(r'(\bnamespace(\s+\w+)?|extern\s+"")\s*$', re.sub(r'"[^"]*"', '""', text[start:at])):
                start = at + 1
                continue
            depth += 1
        elif c == "}":
            if depth == 0:   # a namespace's end
                start = at + 1
                continue
            depth -= 1
        if depth == 0 and c in "};":
            part = text[start:at + 1]
            start = at + 1
            head = re.sub(r"__(launch_bounds|align|grid_constant)__\s*(\((?:[^()]|\([^()]*\))*\))?|template\s*<[^{}]*?>\s*(?=[\w_])", " ", part.split("{")[0])
            name = re.search(r"\bstruct\s+(\w+)", head) or re.search(r"(\w+)\s*\(", head)
            if "{" in part and name:
                found.append((name.group(1), part))
    return found


def test_no_read_only_loads():
    parts = [d for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))) for d in definitions(f)]
    kernels = [d for d in parts if "__global__" in d[1] and "grid_dependency_wait" in d[1]]
    assert len(kernels) >= 15 and any(n == "mc2_gemm_kernel" for n, _ in kernels) and any(n == "a2a_prologue_kernel" for n, _ in kernels)
    reached, todo = {}, list(kernels)
    while todo:
        name, text = todo.pop()
        if id(text) in reached:
            continue
        reached[id(text)] = (name, text)
        words = set(re.findall(r"\w+", text))
        todo += [d for d in parts if d[0] in words and "__global__" not in d[1] and id(d[1]) not in reached]
    assert any(n == "load_weights" for n, _ in reached.values())
    bad = sorted({n for n, t in reached.values() if READ_ONLY.search(t) and n != "load_settled"})
    assert not bad, f"read-only loads in {bad}"


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1500, 40])   # the tiles, and the kernel of few rows
@pytest.mark.parametrize("which", ["int8 product", "product", "norm", "all-to-all"])
def test_inputs_written_by_the_kernel_before(which, m):
    """Biases, weights and codes that one of the library's kernels, whose end the next call's kernel does not wait for to
    begin, writes right before that call."""
    g = torch.Generator().manual_seed(0)

    def t16(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()

    n, k, one = 2048, 512, torch.ones(1, device="cuda")
    steps = [(torch.randint(-127, 128, (1, n), generator=g, dtype=torch.int8).cuda(), one * (i + 1) / 64, t16(k, n)) for i in range(24)]
    kept = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.zeros(k, n, dtype=torch.int8, device="cuda"), torch.zeros(k, device="cuda")
    x, w, y, columns = t16(m, k), t16(n, k, std=k ** -0.5), t16(m, n), torch.rand(n, generator=g).cuda()
    qx, qw, chunks = mc2.mc2_act_quant(x), mc2.mc2_act_quant(w), list(t16(2 * m, k // 2).chunk(2))
    call = {
        "int8 product": lambda v, c: mc2.mc2_quant_matmul(*qx, *qw, bias=v),
        "product": lambda v, c: mc2.mc2_matmul_bias_act(x, w, bias=v)[0],
        "norm": lambda v, c: mc2.mc2_add_rms_norm(y, v)["out"],
        "all-to-all": lambda v, c: mc2.mc2_alltoall_quant_mm(chunks, c, columns, v, x1_quant_mode=mc2.QUANT_PERTOKEN_DYNAMIC)["out"],
    }[which]
    got = []
    for q, s, z in steps:
        mc2.mc2_act_dequant(q, s, out=kept)
        mc2.mc2_act_quant(z, q=codes, scale=scales)
        if which != "all-to-all":   # (whose codes are written last)
            mc2.mc2_act_dequant(q, s, out=kept)
        got.append(call(kept[0], codes))
    torch.cuda.synchronize()
    for (q, s, z), o in zip(steps, got):
        v, c = (q.float() * s)[0].to(torch.bfloat16), mc2.mc2_act_quant(z)[0]
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int16), call(v, c).view(torch.int16))
