"""The calls around the linears without a GPU: each violated constraint is
refused with its status before anything is launched, at the C boundary and in
the Python binding."""
import ctypes

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

FAKE = 0x10000   # aligned and never dereferenced


def norm(x=FAKE, ldx=64, res=FAKE, ldr=64, w=FAKE, wt=mc2.MC2_BF16, m=4, h=64, eps=1e-6, dt=mc2.MC2_BF16, out=FAKE * 2,
         ldo=64, ro=FAKE * 3, ldro=64, rstd=None, mode=0, qd=mc2.MC2_I8, q=None, scale=None):
    return mc2.lib().mc2_add_rms_norm(x, ldx, res, ldr, w, wt, m, h, eps, dt, out, ldo, ro, ldro, rstd, mode, qd, q,
                                      scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), mc2.MC2_ERR_NULL),
    (dict(w=None), mc2.MC2_ERR_NULL),
    (dict(out=None), mc2.MC2_ERR_NULL),
    (dict(m=0), mc2.MC2_ERR_SHAPE),
    (dict(h=0), mc2.MC2_ERR_SHAPE),
    (dict(m=2 ** 31), mc2.MC2_ERR_SHAPE),
    (dict(h=2 ** 30 + 1), mc2.MC2_ERR_SHAPE),
    (dict(eps=-1.0), mc2.MC2_ERR_SHAPE),
    (dict(eps=float("nan")), mc2.MC2_ERR_SHAPE),
    (dict(eps=float("inf")), mc2.MC2_ERR_SHAPE),
    (dict(dt=mc2.MC2_I8), mc2.MC2_ERR_DTYPE),
    (dict(wt=mc2.MC2_F16), mc2.MC2_ERR_DTYPE),
    (dict(ldx=63), mc2.MC2_ERR_SHAPE),
    (dict(ldr=0), mc2.MC2_ERR_SHAPE),
    (dict(ldo=-64), mc2.MC2_ERR_SHAPE),
    (dict(ldro=1), mc2.MC2_ERR_SHAPE),
    (dict(ldx=2 ** 62), mc2.MC2_ERR_SHAPE),
    (dict(x=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
    (dict(rstd=FAKE + 2), mc2.MC2_ERR_UNSUPPORTED),
    (dict(res=None), mc2.MC2_ERR_SHAPE),                  # residual_out without a residual
    (dict(ro=FAKE * 2), mc2.MC2_ERR_SHAPE),               # out and residual_out in one buffer
    (dict(q=FAKE), mc2.MC2_ERR_SHAPE),                    # codes without a mode
    (dict(mode=3), mc2.MC2_ERR_DTYPE),
    (dict(mode=7), mc2.MC2_ERR_NULL),
    (dict(mode=7, q=FAKE), mc2.MC2_ERR_NULL),
    (dict(mode=7, q=FAKE, scale=FAKE, qd=mc2.MC2_BF16), mc2.MC2_ERR_DTYPE),
    (dict(mode=6, q=FAKE, scale=FAKE, qd=mc2.MC2_I8), mc2.MC2_ERR_DTYPE),
    (dict(mode=4, q=FAKE, scale=FAKE + 2), mc2.MC2_ERR_UNSUPPORTED),
])
def test_norm_rejects(kw, status):
    assert norm(**kw) == status
    assert mc2.last_error() != ""


def norm_grad(dy=FAKE, lddy=64, x=FAKE, ldx=64, w=FAKE, wt=mc2.MC2_BF16, rstd=FAKE, dres=FAKE, lddr=64, m=4, h=64,
              dt=mc2.MC2_BF16, dx=FAKE, lddx=64, dw=FAKE, ws=FAKE, nbytes=1 << 20):
    return mc2.lib().mc2_rms_norm_grad(dy, lddy, x, ldx, w, wt, rstd, dres, lddr, m, h, dt, dx, lddx, dw, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), mc2.MC2_ERR_NULL), (dict(x=None), mc2.MC2_ERR_NULL), (dict(w=None), mc2.MC2_ERR_NULL),
    (dict(rstd=None), mc2.MC2_ERR_NULL), (dict(dx=None), mc2.MC2_ERR_NULL),
    (dict(m=0), mc2.MC2_ERR_SHAPE), (dict(h=-1), mc2.MC2_ERR_SHAPE),
    (dict(lddy=8), mc2.MC2_ERR_SHAPE), (dict(lddr=8), mc2.MC2_ERR_SHAPE), (dict(lddx=8), mc2.MC2_ERR_SHAPE),
    (dict(dt=mc2.MC2_E8M0), mc2.MC2_ERR_DTYPE), (dict(wt=mc2.MC2_F16), mc2.MC2_ERR_DTYPE),
    (dict(dy=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED), (dict(rstd=FAKE + 2), mc2.MC2_ERR_UNSUPPORTED),
    (dict(ws=None), mc2.MC2_ERR_WORKSPACE), (dict(nbytes=64), mc2.MC2_ERR_WORKSPACE),
    (dict(ws=FAKE + 4), mc2.MC2_ERR_UNSUPPORTED),
])
def test_norm_grad_rejects(kw, status):
    assert norm_grad(**kw) == status
    assert mc2.last_error() != ""


def test_norm_grad_workspace_query():
    small, large = mc2.mc2_rms_norm_grad_workspace(1, 64), mc2.mc2_rms_norm_grad_workspace(10 ** 6, 64)
    assert 0 < small <= large
    assert mc2.lib().mc2_rms_norm_grad_workspace(1, 64, None) == mc2.MC2_ERR_NULL
    assert mc2.lib().mc2_rms_norm_grad_workspace(0, 64, ctypes.byref(ctypes.c_size_t())) == mc2.MC2_ERR_SHAPE


def linear(x=FAKE, ldx=64, w=FAKE, ldw=64, nk=1, m=4, n=32, k=64, bias=None, act=1, res=FAKE, ldr=32, dt=mc2.MC2_BF16,
           out=FAKE * 2, ldo=32, pre=None, ldp=32):
    return mc2.lib().mc2_matmul_bias_act(x, ldx, w, ldw, nk, m, n, k, bias, act, res, ldr, dt, out, ldo, pre, ldp, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), mc2.MC2_ERR_NULL), (dict(w=None), mc2.MC2_ERR_NULL), (dict(out=None), mc2.MC2_ERR_NULL),
    (dict(m=0), mc2.MC2_ERR_SHAPE), (dict(n=0), mc2.MC2_ERR_SHAPE), (dict(k=0), mc2.MC2_ERR_SHAPE),
    (dict(m=2 ** 31), mc2.MC2_ERR_SHAPE),
    (dict(dt=mc2.MC2_F32), mc2.MC2_ERR_DTYPE), (dict(act=5), mc2.MC2_ERR_DTYPE), (dict(act=-1), mc2.MC2_ERR_DTYPE),
    (dict(ldx=63), mc2.MC2_ERR_SHAPE), (dict(ldw=63), mc2.MC2_ERR_SHAPE), (dict(nk=0, ldw=31), mc2.MC2_ERR_SHAPE),
    (dict(ldr=31), mc2.MC2_ERR_SHAPE), (dict(ldo=31), mc2.MC2_ERR_SHAPE), (dict(pre=FAKE * 4, ldp=31), mc2.MC2_ERR_SHAPE),
    (dict(pre=FAKE * 2), mc2.MC2_ERR_SHAPE), (dict(pre=FAKE), mc2.MC2_ERR_SHAPE),
    (dict(x=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED), (dict(bias=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
])
def test_linear_rejects(kw, status):
    assert linear(**kw) == status
    assert mc2.last_error() != ""


def act_grad_mm(dy=FAKE, lddy=32, w=FAKE, ldw=64, nk=1, z=FAKE, ldz=64, act=1, m=4, n=32, k=64, dt=mc2.MC2_BF16,
                dz=FAKE, lddz=64):
    return mc2.lib().mc2_matmul_act_grad(dy, lddy, w, ldw, nk, z, ldz, act, m, n, k, dt, dz, lddz, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), mc2.MC2_ERR_NULL), (dict(w=None), mc2.MC2_ERR_NULL), (dict(z=None), mc2.MC2_ERR_NULL),
    (dict(dz=None), mc2.MC2_ERR_NULL), (dict(m=0), mc2.MC2_ERR_SHAPE), (dict(act=9), mc2.MC2_ERR_DTYPE),
    (dict(dt=mc2.MC2_F32), mc2.MC2_ERR_DTYPE), (dict(lddy=31), mc2.MC2_ERR_SHAPE), (dict(ldw=63), mc2.MC2_ERR_SHAPE),
    (dict(nk=0, ldw=31), mc2.MC2_ERR_SHAPE), (dict(ldz=63), mc2.MC2_ERR_SHAPE), (dict(lddz=63), mc2.MC2_ERR_SHAPE),
    (dict(z=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
])
def test_act_grad_product_rejects(kw, status):
    assert act_grad_mm(**kw) == status
    assert mc2.last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), mc2.MC2_ERR_NULL), (dict(n=0), mc2.MC2_ERR_SHAPE), (dict(act=7), mc2.MC2_ERR_DTYPE),
    (dict(dt=mc2.MC2_F32), mc2.MC2_ERR_DTYPE), (dict(ldz=7), mc2.MC2_ERR_SHAPE), (dict(dz=FAKE + 1), mc2.MC2_ERR_UNSUPPORTED),
])
def test_act_grad_rejects(kw, status):
    a = dict(dy=FAKE, lddy=8, z=FAKE, ldz=8, act=1, m=4, n=8, dt=mc2.MC2_BF16, dz=FAKE, lddz=8) | kw
    assert mc2.lib().mc2_act_grad(a["dy"], a["lddy"], a["z"], a["ldz"], a["act"], a["m"], a["n"], a["dt"], a["dz"],
                                  a["lddz"], None) == status
    assert mc2.last_error() != ""


# ------------------------------------------------------------------ the binding

B = torch.bfloat16


def refuses(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors: the shape and dtype checks come before the device's")
def test_binding_checks_before_the_library():
    x, w = torch.zeros(4, 64, dtype=B), torch.ones(64, dtype=B)
    f = mc2.mc2_add_rms_norm
    refuses("weight must have shape", f, x, w[:63])
    refuses("residual must have shape", f, x, w, residual=x[:3])
    refuses("residual must be of dtype", f, x, w, residual=x.float())
    refuses("at least 2 dimensions", f, x[0], w)
    refuses("rows of adjacent elements", f, torch.zeros(64, 4, dtype=B).t(), w)
    refuses("rows of adjacent elements", f, torch.zeros(1, 64, dtype=B).expand(4, 64), w)
    refuses("rows of adjacent elements", f, torch.zeros(4, 4, 128, dtype=B)[:, :3, :64], w)
    refuses("q_dtype must be", f, x, w, quant_mode=mc2.QUANT_MX, q_dtype=torch.int32)
    refuses("scale must have shape", f, x, w, quant_mode=mc2.QUANT_MX, q_dtype=torch.float8_e4m3fn,
            scale=torch.zeros(4, 3, dtype=torch.uint8))
    refuses("need a quant_mode", f, x, w, q=torch.zeros(4, 64, dtype=torch.int8))
    refuses("no CUDA device", f, x, w)
    g = mc2.mc2_rms_norm_grad
    refuses("rstd must have shape", g, x, x, w, torch.zeros(5))
    refuses("dw must be of dtype", g, x, x, w, torch.zeros(4), dw=torch.zeros(64))
    refuses("no CUDA device", g, x, x, w, torch.zeros(4))
    l = mc2.mc2_matmul_bias_act
    refuses("activation must be one of", l, x, torch.zeros(8, 64, dtype=B), activation="swish")
    refuses("w must have shape", l, x, torch.zeros(8, 63, dtype=B))
    refuses("w must have 2 dimensions", l, x, w)
    refuses("w must be of dtype", l, x, torch.zeros(8, 64))
    refuses("bias must have shape", l, x, torch.zeros(8, 64, dtype=B), bias=torch.zeros(7, dtype=B))
    refuses("residual must have shape", l, x, torch.zeros(8, 64, dtype=B), residual=x)
    refuses("no CUDA device", l, x, torch.zeros(8, 64, dtype=B))
    refuses("z must have shape", mc2.mc2_matmul_act_grad, x, torch.zeros(64, 8, dtype=B), x, activation="relu")
    refuses("z must be of dtype", mc2.mc2_act_grad, x, x.float(), activation="relu")
