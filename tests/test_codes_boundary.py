"""The calls on 8-bit codes without a GPU: each violated constraint is refused with its status before anything is
launched, at the C boundary and in the Python binding."""
import ctypes

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

FAKE = 0x10000   # aligned and never dereferenced
B = torch.bfloat16
BIG = 2 ** 30 + 1


def product(x=FAKE, ldx=64, xs=FAKE, w=FAKE, ldw=64, nk=1, ws=FAKE, m=400, n=32, k=64, bias=None, bt=mc2.MC2_BF16, act=1, res=None,
            ldr=32, dt=mc2.MC2_BF16, out=FAKE * 2, ldo=32, wk=FAKE, nbytes=1 << 40):
    return mc2.lib().mc2_quant_matmul(x, ldx, xs, w, ldw, nk, ws, m, n, k, bias, bt, act, res, ldr, dt, out, ldo, wk, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), mc2.MC2_ERR_NULL), (dict(xs=None), mc2.MC2_ERR_NULL), (dict(w=None), mc2.MC2_ERR_NULL),
    (dict(ws=None), mc2.MC2_ERR_NULL), (dict(out=None), mc2.MC2_ERR_NULL),
    (dict(m=0), mc2.MC2_ERR_SHAPE), (dict(n=0), mc2.MC2_ERR_SHAPE), (dict(k=0), mc2.MC2_ERR_SHAPE), (dict(m=-1), mc2.MC2_ERR_SHAPE),
    (dict(m=BIG), mc2.MC2_ERR_SHAPE), (dict(n=BIG), mc2.MC2_ERR_SHAPE),
    (dict(k=131072, ldx=131072, ldw=131072), mc2.MC2_ERR_SHAPE),
    (dict(dt=mc2.MC2_F32), mc2.MC2_ERR_DTYPE), (dict(dt=mc2.MC2_I8), mc2.MC2_ERR_DTYPE),
    (dict(act=5), mc2.MC2_ERR_DTYPE), (dict(act=-1), mc2.MC2_ERR_DTYPE),
    (dict(bias=FAKE, bt=mc2.MC2_F16), mc2.MC2_ERR_DTYPE), (dict(bias=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
    (dict(bias=FAKE + 2, bt=mc2.MC2_F32), mc2.MC2_ERR_UNSUPPORTED),
    (dict(ldx=63), mc2.MC2_ERR_SHAPE), (dict(ldw=63), mc2.MC2_ERR_SHAPE), (dict(nk=0, ldw=31), mc2.MC2_ERR_SHAPE),
    (dict(ldo=31), mc2.MC2_ERR_SHAPE), (dict(res=FAKE, ldr=31), mc2.MC2_ERR_SHAPE), (dict(ldx=2 ** 61), mc2.MC2_ERR_SHAPE),
    (dict(res=FAKE * 2, ldr=40), mc2.MC2_ERR_SHAPE),      # in place, but with another stride
    (dict(xs=FAKE + 2), mc2.MC2_ERR_UNSUPPORTED), (dict(ws=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED), (dict(out=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
])
def test_product_rejects(kw, status):
    assert product(**kw) == status
    assert mc2.last_error() != ""


def quant(z=FAKE, ldz=64, m=4, h=64, act=0, dt=mc2.MC2_BF16, mode=7, qd=mc2.MC2_I8, q=FAKE, scale=FAKE):
    return mc2.lib().mc2_act_quant(z, ldz, m, h, act, dt, mode, qd, q, scale, None)


def dequant(q=FAKE, scale=FAKE, m=4, h=64, act=0, mode=7, qd=mc2.MC2_I8, dt=mc2.MC2_BF16, out=FAKE, ldo=64):
    return mc2.lib().mc2_act_dequant(q, scale, m, h, act, mode, qd, dt, out, ldo, None)


def grad(dy=FAKE, lddy=64, q=FAKE, scale=FAKE, m=4, h=64, act=1, mode=7, qd=mc2.MC2_I8, dt=mc2.MC2_BF16, dz=FAKE * 2, lddz=64):
    return mc2.lib().mc2_act_grad_quant(dy, lddy, q, scale, m, h, act, mode, qd, dt, dz, lddz, None)


def weight(dy=FAKE, lddy=32, q=FAKE, scale=FAKE, m=4, n=32, h=64, act=0, mode=7, qd=mc2.MC2_I8, dt=mc2.MC2_BF16, dw=FAKE, db=None,
           wk=FAKE, nbytes=1 << 40):
    return mc2.lib().mc2_matmul_weight_grad_quant(dy, lddy, q, scale, m, n, h, act, mode, qd, dt, dw, db, wk, nbytes, None)


KEPT = [(dict(q=None), mc2.MC2_ERR_NULL), (dict(scale=None), mc2.MC2_ERR_NULL), (dict(m=0), mc2.MC2_ERR_SHAPE), (dict(h=0), mc2.MC2_ERR_SHAPE),
        (dict(m=BIG), mc2.MC2_ERR_SHAPE), (dict(h=BIG), mc2.MC2_ERR_SHAPE), (dict(act=5), mc2.MC2_ERR_DTYPE), (dict(act=-1), mc2.MC2_ERR_DTYPE),
        (dict(mode=0), mc2.MC2_ERR_DTYPE), (dict(mode=3), mc2.MC2_ERR_DTYPE), (dict(qd=mc2.MC2_BF16), mc2.MC2_ERR_DTYPE),
        (dict(mode=6), mc2.MC2_ERR_DTYPE), (dict(scale=FAKE + 2), mc2.MC2_ERR_UNSUPPORTED), (dict(mode=4, scale=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
        (dict(dt=mc2.MC2_I8), mc2.MC2_ERR_DTYPE)]


@pytest.mark.parametrize("call", [quant, dequant, grad, weight])
@pytest.mark.parametrize("kw,status", KEPT)
def test_codes_reject(call, kw, status):
    assert call(**kw) == status
    assert mc2.last_error() != ""


@pytest.mark.parametrize("call,kw,status", [
    (quant, dict(z=None), mc2.MC2_ERR_NULL), (quant, dict(ldz=63), mc2.MC2_ERR_SHAPE), (quant, dict(z=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
    (quant, dict(z=FAKE + 2, dt=mc2.MC2_F32), mc2.MC2_ERR_UNSUPPORTED), (quant, dict(ldz=2 ** 61), mc2.MC2_ERR_SHAPE),
    (dequant, dict(out=None), mc2.MC2_ERR_NULL), (dequant, dict(ldo=63), mc2.MC2_ERR_SHAPE), (dequant, dict(out=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
    (grad, dict(dy=None), mc2.MC2_ERR_NULL), (grad, dict(dz=None), mc2.MC2_ERR_NULL), (grad, dict(lddy=63), mc2.MC2_ERR_SHAPE),
    (grad, dict(lddz=63), mc2.MC2_ERR_SHAPE), (grad, dict(dz=FAKE, lddz=72), mc2.MC2_ERR_SHAPE), (grad, dict(dt=mc2.MC2_F32), mc2.MC2_ERR_DTYPE),
    (weight, dict(dy=None), mc2.MC2_ERR_NULL), (weight, dict(dw=None), mc2.MC2_ERR_NULL), (weight, dict(n=0), mc2.MC2_ERR_SHAPE),
    (weight, dict(lddy=31), mc2.MC2_ERR_SHAPE), (weight, dict(dy=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED), (weight, dict(dw=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
    (weight, dict(db=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED), (weight, dict(dt=mc2.MC2_F32), mc2.MC2_ERR_DTYPE),
])
def test_each_call_rejects(call, kw, status):
    assert call(**kw) == status
    assert mc2.last_error() != ""


def test_workspace_queries():
    L, n = mc2.lib(), ctypes.c_size_t(1)
    ref = ctypes.byref(n)
    f = L.mc2_quant_matmul_workspace
    good = (FAKE, 4096, FAKE, 4096, 1, 4096, 4096, 4096, None, 0, FAKE, 4096, ref)
    assert f(*good) == mc2.MC2_OK and n.value >= 2 * 2 * 4096 * 4096   # both operands in 16 bits
    few = (*good[:5], 16, *good[6:])
    assert f(*few) == mc2.MC2_OK and n.value == 0
    # an operand that does not begin at 16 bytes goes through it
    assert f(FAKE + 1, *few[1:]) == mc2.MC2_OK and 16 * 4096 <= n.value < 4096 * 4096
    assert f(*few[:2], FAKE + 8, *few[3:]) == mc2.MC2_OK and n.value >= 4096 * 4096
    for at, value, status in ((0, None, mc2.MC2_ERR_NULL), (2, None, mc2.MC2_ERR_NULL), (10, None, mc2.MC2_ERR_NULL), (12, None, mc2.MC2_ERR_NULL),
                              (5, 0, mc2.MC2_ERR_SHAPE), (1, 8, mc2.MC2_ERR_SHAPE), (11, 31, mc2.MC2_ERR_SHAPE)):
        assert f(*good[:at], value, *good[at + 1:]) == status
    f = L.mc2_matmul_weight_grad_quant_workspace
    good = (FAKE, 32, FAKE, 4, 32, 64, ref)
    assert f(*good) == mc2.MC2_OK and n.value > 0
    for at, value, status in ((0, None, mc2.MC2_ERR_NULL), (2, None, mc2.MC2_ERR_NULL), (6, None, mc2.MC2_ERR_NULL), (5, 0, mc2.MC2_ERR_SHAPE),
                              (1, 31, mc2.MC2_ERR_SHAPE)):
        assert f(*good[:at], value, *good[at + 1:]) == status


@pytest.mark.parametrize("kw", [dict(wk=None), dict(nbytes=64)])
def test_a_workspace_that_is_missing_or_small(kw):
    many = dict(m=4096, n=4096, k=4096, ldx=4096, ldw=4096, ldo=4096)
    assert product(**many, **kw) == mc2.MC2_ERR_WORKSPACE
    assert weight(**kw) == mc2.MC2_ERR_WORKSPACE
    assert product(**many, wk=FAKE + 8) == mc2.MC2_ERR_UNSUPPORTED and weight(wk=FAKE + 8) == mc2.MC2_ERR_UNSUPPORTED


def refuses(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors: the shape and dtype checks come before the device's")
def test_binding_checks_before_the_library():
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    w, ws = torch.zeros(32, 64, dtype=torch.int8), torch.ones(32)
    f = mc2.mc2_quant_matmul
    refuses("x must be of dtype", f, q.float(), s, w, ws)
    refuses("x_scale must have shape", f, q, s[:3], w, ws)
    refuses("x_scale must be of dtype", f, q, s.double(), w, ws)
    refuses("w must have shape", f, q, s, w[:, :63], ws)
    refuses("w must have 2 dimensions", f, q, s, ws, ws)
    refuses("w_scale must have shape", f, q, s, w, ws[:31])
    refuses("bias must have shape", f, q, s, w, ws, bias=ws[:31])
    refuses("bias must be of dtype", f, q, s, w, ws, bias=ws.half())
    refuses("residual must have shape", f, q, s, w, ws, residual=torch.zeros(4, 31, dtype=B))
    refuses("residual must be of dtype", f, q, s, w, ws, residual=torch.zeros(4, 32, dtype=B), dtype=torch.float16)
    refuses("unsupported dtype", f, q, s, w, ws, dtype=torch.float64)
    refuses("activation must be one of", f, q, s, w, ws, activation="swish")
    refuses("at least 2 dimensions", f, q[0], s, w, ws)
    refuses("no CUDA device", f, q, s, w, ws)
    z = torch.zeros(4, 64, dtype=B)
    a = mc2.mc2_act_quant
    refuses("q_dtype must be", a, z, q_dtype=torch.uint8)
    refuses("at least 2 dimensions", a, z[0])
    refuses("q must have shape", a, z, q=q[:3])
    refuses("scale must have shape", a, z, quant_mode=mc2.QUANT_PERGROUP, scale=s)
    refuses("rows of adjacent elements", a, z.t())
    d = mc2.mc2_act_dequant
    refuses("q must be of dtype", d, z, s)
    refuses("scale must have shape", d, q, s[:3])
    refuses("scale must have shape", d, q, torch.ones(4, 2))
    refuses("scale must have shape", d, q, torch.ones(4, 3, dtype=torch.uint8))
    refuses("scale must be of dtype", d, q, s.half())
    refuses("out must have shape", d, q, s, out=z[:3])
    refuses("dy must have shape", mc2.mc2_act_grad_quant, z[:3], q, s, activation="relu")
    refuses("dz must be of dtype", mc2.mc2_act_grad_quant, z, q, s, activation="relu", dz=z.float())
    g = mc2.mc2_matmul_weight_grad_quant
    refuses("dy must have shape", g, z[:3], q, s)
    refuses("dw must have shape", g, z, q, s, dw=z)
    refuses("db must be of dtype", g, z, q, s, db=torch.zeros(64))
    refuses("no CUDA device", d, q, s)
