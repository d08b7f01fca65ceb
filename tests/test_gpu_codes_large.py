"""Products of 8-bit codes whose matrices have more than 2^32 elements: the last rows and columns are those of a small call."""
import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
LONG = 540000   # rows of 8192 codes: 4.4e9


def codes(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-127, 128, (rows, cols), generator=g, dtype=torch.int8, device="cuda")


def scales(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(n, generator=g, device="cuda") + 0.5) / 512


def exact(x, xs, w, ws):
    return ((x.double() @ w.double().t()).float() * xs[:, None] * ws).to(BF16)


@pytest.mark.parametrize("m", [1, 3, 40, 100])
def test_a_weight_of_many_rows(m):
    x, xs, w, ws = codes(m, 8192, 1), scales(m, 2), codes(LONG, 8192, 3), scales(LONG, 4)
    out = mc2.mc2_quant_matmul(x, xs, w, ws)
    for a in (0, LONG // 2 - 100, LONG - 300):
        assert torch.equal(out[:, a:a + 300], exact(x, xs, w[a:a + 300], ws[a:a + 300])), a


@pytest.mark.parametrize("m", [40, 100])
def test_a_weight_of_many_columns(m):
    x, xs, w, ws = codes(m, 8192, 1), scales(m, 2), codes(8192, LONG, 3), scales(LONG, 4)
    out = mc2.mc2_quant_matmul(x, xs, w, ws, w_is_nk=False)
    for a in (0, LONG // 2 - 100, LONG - 300):
        assert torch.equal(out[:, a:a + 300], exact(x, xs, w[:, a:a + 300].t(), ws[a:a + 300])), a


@pytest.mark.parametrize("n", [72, 73])   # an output that tensor copies write, and one that they do not
def test_many_tokens(n):
    x, xs, w, ws = codes(LONG, 8192, 1), scales(LONG, 2), codes(n, 8192, 3), scales(n, 4)
    res = torch.randn(LONG, n, device="cuda").to(BF16)
    out = mc2.mc2_quant_matmul(x, xs, w, ws, residual=res)
    for a in (0, LONG // 2 - 100, LONG - 300):
        s = slice(a, a + 300)
        z = (x[s].double() @ w.double().t()).float() * xs[s, None] * ws + res[s].float()
        assert torch.equal(out[s], z.to(BF16)), a


def test_many_outputs():
    m, n, k = 66008, 66000, 128
    x, xs, w, ws = codes(m, k, 1), scales(m, 2), codes(n, k, 3), scales(n, 4)
    out = mc2.mc2_quant_matmul(x, xs, w, ws)
    for a in (0, m // 2, m - 200):
        assert torch.equal(out[a:a + 200, -200:], exact(x[a:a + 200], xs[a:a + 200], w[-200:], ws[-200:])), a


@pytest.mark.parametrize("n", [64, 65])
def test_weight_gradient_of_many_tokens(n):
    """Ones at a few tokens: the sums are those tokens' codes."""
    q, s = codes(LONG, 8192, 1), torch.ones(LONG, device="cuda") / 64
    dy = torch.zeros(LONG, n, dtype=BF16, device="cuda")
    at = [0, 7, LONG // 2, LONG - 1]
    for i, t in enumerate(at):
        dy[t, 16 * i] = 1
    dw, db = mc2.mc2_matmul_weight_grad_quant(dy, q, s)
    for i, t in enumerate(at):
        assert torch.equal(dw[16 * i], (q[t].float() / 64).to(BF16)) and db[16 * i] == 1
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[[16 * i for i in range(4)]] = False
    assert not dw[rest].any() and not db[rest].any()


@pytest.mark.parametrize("k", [66008, 66001])
def test_weight_gradient_of_many_outputs(k):
    m, n = 24, 66000
    q, s = codes(m, k, 1), torch.ones(m, device="cuda") / 64
    dy = torch.zeros(m, n, dtype=BF16, device="cuda")
    dy[torch.arange(n) % m, torch.arange(n)] = 2
    dw, db = mc2.mc2_matmul_weight_grad_quant(dy, q, s)
    for a in (0, n // 2, n - 500):
        i = torch.arange(a, a + 500)
        assert torch.equal(dw[a:a + 500], (q[(i % m).cuda()].float() / 32).to(BF16)), a
    assert (db == 2).all()
