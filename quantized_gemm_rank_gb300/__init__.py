"""GB300 (sm_103a) MC2 fused linears: Python binding of the C ABI in
``include/mc2_gb300.h``.

Argument marshalling only: every step of the operations runs in the CUDA
library ``libmc2_gb300.so`` (built in-tree by :mod:`.build`).  The calls around
the linears marshal their regular case in an extension module (``binding/native.cpp``).  PyTorch
provides device memory and streams.  There is no CPU fallback: if the library
cannot be built or loaded, importing the functions raises.

  mc2_all_gather_mm        out = concat_m(x_chunks) @ x2 (+ bias), plus gathered
  mc2_alltoall_quant_mm    out = (Quant(permute(chunks)) @ x2) * x1s * x2s + bias
  mc2_matmul_reduce_scatter  out_j = (sum_r X_r @ W_r^T)[rows of rank j] (+ bias)
  mc2_matmul_weight_grad   dw = dy^T @ x, db = dy.sum(0)
  mc2_quant_all_reduce     out = sum_r dequant(x_r, scales_r)  (int8/fp8 codes)

and, around the linears:

  mc2_add_rms_norm         out = rmsnorm(x + residual) * weight, and its 8-bit codes with scales
  mc2_rms_norm_grad        its gradient
  mc2_matmul_bias_act      out = act(x @ w^T + bias) + residual
  mc2_matmul_act_grad      dz = (dy @ w) * act'(z)
  mc2_act_grad             dz = dy * act'(z)

and on 8-bit codes with their scales:

  mc2_quant_matmul         out = act(x @ w^T * x_scale * w_scale + bias) + residual, int8 by int8
  mc2_act_quant            the codes of act(z)
  mc2_act_dequant          act of what codes stand for
  mc2_act_grad_quant       dz = dy * act'(z), z kept in 8 bits
  mc2_matmul_weight_grad_quant  dw = dy^T @ act(x), db = dy.sum(0), x kept in 8 bits
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from typing import Optional, Sequence

import torch

from . import build as _build

MC2_OK = 0
MC2_ERR_NULL = -1
MC2_ERR_SHAPE = -2
MC2_ERR_DTYPE = -3
MC2_ERR_UNSUPPORTED = -4
MC2_ERR_WORKSPACE = -5
MC2_ERR_CUDA = -6
MC2_ERR_TIMEOUT = -7

MC2_F16, MC2_BF16, MC2_F32, MC2_I8 = 1, 2, 3, 4
MC2_F8E4M3, MC2_F8E5M2, MC2_E8M0 = 5, 6, 7
QUANT_NONE = 0
QUANT_PERCHANNEL = 2
QUANT_PERTOKEN = 3
QUANT_PERGROUP = 4
QUANT_MX = 6
QUANT_PERTOKEN_DYNAMIC = 7

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_lib = None


class Mc2Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_str(status)}: {message}")
        self.status = status
        self.message = message


def lib() -> ctypes.CDLL:
    """Load (building first if the sources changed) the CUDA library."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        L.mc2_all_gather_mm.argtypes = [_P, _INT, _I64, _I64, _P, _I64, _INT, _P, _INT, _INT, _P, _P, _P]
        L.mc2_all_gather_mm.restype = _INT
        L.mc2_matmul_reduce_scatter.argtypes = [_P, _P, _INT, _I64, _I64, _I64, _INT, _P, _INT, _P, _P]
        L.mc2_matmul_reduce_scatter.restype = _INT
        L.mc2_matmul_weight_grad.argtypes = [_P, _I64, _I64, _P, _I64, _INT, _P, _P, _P]
        L.mc2_matmul_weight_grad.restype = _INT
        L.mc2_quant_all_reduce.argtypes = [_P, _P, _INT, _I64, _I64, _INT, _INT, _INT, _P, _P]
        L.mc2_quant_all_reduce.restype = _INT
        L.mc2_alltoall_quant_mm_workspace.argtypes = [_INT, _I64, _I64, _I64, _INT, _INT,
                                                      ctypes.POINTER(ctypes.c_size_t)]
        L.mc2_alltoall_quant_mm_workspace.restype = _INT
        L.mc2_alltoall_quant_mm.argtypes = [_P, _INT, _I64, _I64, _INT, _P, _P, _P, _P, _INT, _INT, _INT, _I64,
                                            _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.mc2_alltoall_quant_mm.restype = _INT
        L.mc2_alltoall_quant_mm_no_alloc.argtypes = [_P, _INT, _I64, _I64, _INT, _P, _P, _P, _P, _INT, _INT, _INT,
                                                     _I64, _P, _P, _P, _P, _P, _P]
        L.mc2_alltoall_quant_mm_no_alloc.restype = _INT
        L.mc2_add_rms_norm.argtypes = [_P, _I64, _P, _I64, _P, _INT, _I64, _I64, ctypes.c_float, _INT, _P, _I64,
                                       _P, _I64, _P, _INT, _INT, _P, _P, _P]
        L.mc2_add_rms_norm.restype = _INT
        L.mc2_rms_norm_grad_workspace.argtypes = [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)]
        L.mc2_rms_norm_grad_workspace.restype = _INT
        L.mc2_rms_norm_grad.argtypes = [_P, _I64, _P, _I64, _P, _INT, _P, _P, _I64, _I64, _I64, _INT, _P, _I64,
                                        _P, _P, ctypes.c_size_t, _P]
        L.mc2_rms_norm_grad.restype = _INT
        L.mc2_matmul_bias_act.argtypes = [_P, _I64, _P, _I64, _INT, _I64, _I64, _I64, _P, _INT, _P, _I64, _INT,
                                          _P, _I64, _P, _I64, _P]
        L.mc2_matmul_bias_act.restype = _INT
        L.mc2_matmul_act_grad.argtypes = [_P, _I64, _P, _I64, _INT, _P, _I64, _INT, _I64, _I64, _I64, _INT, _P,
                                          _I64, _P]
        L.mc2_matmul_act_grad.restype = _INT
        L.mc2_act_grad.argtypes = [_P, _I64, _P, _I64, _INT, _I64, _I64, _INT, _P, _I64, _P]
        L.mc2_act_grad.restype = _INT
        L.mc2_quant_matmul_workspace.argtypes = [_P, _I64, _P, _I64, _INT, _I64, _I64, _I64, _P, _I64, _P, _I64,
                                                 ctypes.POINTER(ctypes.c_size_t)]
        L.mc2_quant_matmul_workspace.restype = _INT
        L.mc2_quant_matmul.argtypes = [_P, _I64, _P, _P, _I64, _INT, _P, _I64, _I64, _I64, _P, _INT, _INT, _P, _I64, _INT,
                                       _P, _I64, _P, ctypes.c_size_t, _P]
        L.mc2_quant_matmul.restype = _INT
        L.mc2_act_quant.argtypes = [_P, _I64, _I64, _I64, _INT, _INT, _INT, _INT, _P, _P, _P]
        L.mc2_act_quant.restype = _INT
        L.mc2_act_dequant.argtypes = [_P, _P, _I64, _I64, _INT, _INT, _INT, _INT, _P, _I64, _P]
        L.mc2_act_dequant.restype = _INT
        L.mc2_act_grad_quant.argtypes = [_P, _I64, _P, _P, _I64, _I64, _INT, _INT, _INT, _INT, _P, _I64, _P]
        L.mc2_act_grad_quant.restype = _INT
        L.mc2_matmul_weight_grad_quant_workspace.argtypes = [_P, _I64, _P, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)]
        L.mc2_matmul_weight_grad_quant_workspace.restype = _INT
        L.mc2_matmul_weight_grad_quant.argtypes = [_P, _I64, _P, _P, _I64, _I64, _I64, _INT, _INT, _INT, _INT, _P, _P, _P,
                                                   ctypes.c_size_t, _P]
        L.mc2_matmul_weight_grad_quant.restype = _INT
        L.mc2_status_str.argtypes = [_INT]
        L.mc2_status_str.restype = ctypes.c_char_p
        L.mc2_last_error.argtypes = []
        L.mc2_last_error.restype = ctypes.c_char_p
        L.mc2_device_status.argtypes = []
        L.mc2_device_status.restype = _INT
        L.mc2_set_launch_events.argtypes = [_P, _INT]
        L.mc2_set_launch_events.restype = _INT
        L.mc2_test_expire_next_flag_waits.argtypes = [ctypes.c_uint64]
        L.mc2_test_expire_next_flag_waits.restype = _INT
        _lib = L
    return _lib


_native_module = None


def _native():
    """The extension module of the binding (built first if its source changed)."""
    global _native_module
    if _native_module is None:
        lib()
        path = _build.build_native()
        spec = importlib.util.spec_from_file_location(__name__ + "._native", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native_module = module
    return _native_module


def library_path() -> str:
    return _build.LIB


def status_str(status: int) -> str:
    return lib().mc2_status_str(status).decode()


def last_error() -> str:
    return lib().mc2_last_error().decode()


def _check(status: int):
    if status != MC2_OK:
        raise Mc2Error(status, last_error())


_DTYPE_CODES = {torch.float16: MC2_F16, torch.bfloat16: MC2_BF16, torch.float32: MC2_F32, torch.int8: MC2_I8}


def _dtype_code(dt: torch.dtype) -> int:
    if dt not in _DTYPE_CODES:
        raise ValueError(f"unsupported dtype {dt}")
    return _DTYPE_CODES[dt]


_raw_device = None   # the current device's index, once CUDA is known to be there


def _current_device() -> int:
    """The CUDA device the library launches on, or -1 without CUDA."""
    global _raw_device
    if _raw_device is not None:
        return _raw_device()
    if not torch.cuda.is_available():
        return -1
    cur = torch.cuda.current_device()   # (initialises CUDA, once)
    _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return cur


# Every tensor goes to the library as a bare pointer, and its kernels trust the
# sizes passed beside it, so each tensor is checked first against the shape
# and dtype those sizes imply (a smaller buffer would be read or written past
# its end), against the current device (the library launches there: a tensor
# elsewhere would reach its kernels as a foreign pointer) and for contiguity.
# Without CUDA the device is -1, which a CPU tensor also reports: shape and
# dtype mistakes are then still reported first, and _need_device refuses the
# call before the library is reached.

def _refuse(t: torch.Tensor, shape, dtype, what: str, cur: int):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be of dtype {dtype}, got {t.dtype}")
    if cur < 0 or t.get_device() != cur:
        where = "a CUDA device (none is available)" if cur < 0 else f"the current device (cuda:{cur})"
        raise ValueError(f"{what} must be a CUDA tensor on {where}")
    raise ValueError(f"{what} must be contiguous")


def _arg(t: torch.Tensor, shape, dtype, what: str, cur: int) -> int:
    """The tensor's device pointer, once its shape, dtype, device and layout are right."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != cur or not t.is_contiguous():
        _refuse(t, shape, dtype, what, cur)
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], shape, dtype, what: str, cur: int) -> Optional[int]:
    return None if t is None else _arg(t, shape, dtype, what, cur)


def _args(ts: Sequence[torch.Tensor], shape, dtype, what: str, cur: int):
    """A C array of the tensors' pointers, each checked as by _arg."""
    if len(ts) == 0:
        raise ValueError(f"{what} is empty")
    ptrs = []
    for t in ts:
        if t.shape != shape or t.dtype != dtype or t.get_device() != cur or not t.is_contiguous():
            _refuse(t, shape, dtype, f"{what}[{len(ptrs)}]", cur)
        ptrs.append(t.data_ptr())
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def _need_device(cur: int) -> None:
    if cur < 0:
        raise ValueError("the tensors must be CUDA tensors on the current device, and no CUDA device is available")


_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, cur: int) -> Optional[int]:
    if stream is None:
        if _raw_current_stream is not None:
            # the current stream's handle without building a Stream object (a call's
            # largest single piece of Python-side work)
            return _raw_current_stream(cur)
        stream = torch.cuda.current_stream()
    elif stream.device_index != cur:
        raise ValueError(f"stream must belong to the current device (cuda:{cur})")
    return stream.cuda_stream


def _on_stream(f, args: dict):
    """A call with ``stream=``: f under that stream, whose pool its workspace and new outputs come from.

    (Memory of the current stream's pool could still be in use there, and a
    workspace would go back to it, for the next tensor made, while the launched kernels
    use it.)  The new outputs may be used on the caller's stream, once that waits for the
    given one, and freed like any tensor of its own: their memory is kept until it is done with them.
    (This takes some 20 us of host time; a call within ``torch.cuda.stream(stream)`` takes none of it.)
    """
    stream = args.pop("stream")
    cur = _current_device()
    if cur < 0:
        return f(**args)   # (refuses, in its own words)
    if stream.device_index != cur:
        raise ValueError(f"stream must belong to the current device (cuda:{cur})")
    if _raw_current_stream is not None and stream.cuda_stream == _raw_current_stream(cur):
        return f(**args)
    home = torch.cuda.current_stream()
    torch.cuda.set_stream(stream)   # (the context manager takes 5 us of host time more)
    try:
        r = f(**args)
    finally:
        torch.cuda.set_stream(home)
    given = set()
    for v in args.values():
        given.update(map(id, v) if isinstance(v, (list, tuple)) else (id(v),))
    made = r.values() if isinstance(r, dict) else r if isinstance(r, (list, tuple)) else (r,)
    for t in made:
        if t is not None and id(t) not in given:
            t.record_stream(home)
    return r


def mc2_all_gather_mm(x_chunks: Sequence[torch.Tensor], x2: torch.Tensor, *, x2_is_nk: bool = False,
                      bias: Optional[torch.Tensor] = None, gather_output: bool = True,
                      out: Optional[torch.Tensor] = None, gathered: Optional[torch.Tensor] = None,
                      stream=None):
    """AllGatherMatmul on the rank chunks already resident on this GPU.

    x_chunks: world_size tensors (m_local, k); x2 (k, n), or w (n, k) with
    ``x2_is_nk``.  Returns (out (m, n), gathered (m, k) or None).
    """
    if stream is not None:
        return _on_stream(mc2_all_gather_mm, locals())
    cur = _current_device()
    R = len(x_chunks)
    m_local, k = x_chunks[0].shape
    n = x2.shape[0] if x2_is_nk else x2.shape[1]
    dt = x_chunks[0].dtype
    ptrs = _args(x_chunks, (m_local, k), dt, "x_chunks", cur)
    x2p = _arg(x2, (n, k) if x2_is_nk else (k, n), dt, "x2", cur)
    bp = _opt(bias, (n,), dt, "bias", cur)
    if out is None:
        out = torch.empty((R * m_local, n), dtype=dt, device=x_chunks[0].device)
    outp = _arg(out, (R * m_local, n), dt, "out", cur)
    gp = None
    if gather_output:
        if gathered is None:
            gathered = torch.empty((R * m_local, k), dtype=dt, device=x_chunks[0].device)
        gp = _arg(gathered, (R * m_local, k), dt, "gathered", cur)
    _need_device(cur)
    st = lib().mc2_all_gather_mm(ptrs, R, m_local, k, x2p, n, int(x2_is_nk), bp, _dtype_code(dt), int(gather_output),
                                 outp, gp, _stream(stream, cur))
    _check(st)
    return out, (gathered if gather_output else None)


def mc2_matmul_reduce_scatter(x_chunks: Sequence[torch.Tensor], w_chunks: Sequence[torch.Tensor], *,
                              w_is_nk: bool = True, bias: Optional[torch.Tensor] = None,
                              out_chunks: Optional[Sequence[torch.Tensor]] = None, stream=None):
    """MatmulReduceScatter on the ranks' shards already resident on this GPU.

    x_chunks: world_size tensors (m, k_local); w_chunks: world_size weight shards
    (n, k_local) (or (k_local, n) with ``w_is_nk=False``).  Returns the list of
    the ranks' outputs, each (m / world_size, n).
    """
    if stream is not None:
        return _on_stream(mc2_matmul_reduce_scatter, locals())
    cur = _current_device()
    R = len(x_chunks)
    m, k_local = x_chunks[0].shape
    n = w_chunks[0].shape[0] if w_is_nk else w_chunks[0].shape[1]
    dt = x_chunks[0].dtype
    if len(w_chunks) != R:
        raise ValueError(f"w_chunks must hold {R} shards (one per rank), got {len(w_chunks)}")
    if out_chunks is not None and len(out_chunks) != R:
        raise ValueError(f"out_chunks must hold {R} outputs (one per rank), got {len(out_chunks)}")
    xp = _args(x_chunks, (m, k_local), dt, "x_chunks", cur)
    wp = _args(w_chunks, (n, k_local) if w_is_nk else (k_local, n), dt, "w_chunks", cur)
    bp = _opt(bias, (n,), dt, "bias", cur)
    if out_chunks is None:
        out_chunks = [torch.empty((m // R, n), dtype=dt, device=x_chunks[0].device) for _ in range(R)]
    op = _args(out_chunks, (m // R, n), dt, "out_chunks", cur)
    _need_device(cur)
    st = lib().mc2_matmul_reduce_scatter(xp, wp, R, m, k_local, n, int(w_is_nk), bp, _dtype_code(dt), op,
                                         _stream(stream, cur))
    _check(st)
    return list(out_chunks)


def mc2_matmul_weight_grad(dy: torch.Tensor, x: torch.Tensor, *, with_bias: bool = True,
                           dw: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None, stream=None):
    """dW = dY^T @ X (n, k) and, with ``with_bias``, dB = dY.sum(0) (n).

    dy (m, n) and x (m, k) of one 16-bit type on this GPU (for the all-gather
    layer, x is the ``gathered`` output of its forward call).  Returns (dw, db).
    """
    if stream is not None:
        return _on_stream(mc2_matmul_weight_grad, locals())
    cur = _current_device()
    m, n = dy.shape
    k = x.shape[1]
    dt = dy.dtype
    dyp = _arg(dy, (m, n), dt, "dy", cur)
    xp = _arg(x, (m, k), dt, "x", cur)
    if dw is None:
        dw = torch.empty((n, k), dtype=dt, device=dy.device)
    dwp = _arg(dw, (n, k), dt, "dw", cur)
    dbp = None
    if with_bias:
        if db is None:
            db = torch.empty((n,), dtype=dt, device=dy.device)
        dbp = _arg(db, (n,), dt, "db", cur)
    _need_device(cur)
    st = lib().mc2_matmul_weight_grad(dyp, m, n, xp, k, _dtype_code(dt), dwp, dbp, _stream(stream, cur))
    _check(st)
    return dw, (db if with_bias else None)


_QAR_X = {"int8": MC2_I8, "e4m3": MC2_F8E4M3, "e5m2": MC2_F8E5M2}
_QAR_X_BY_DTYPE = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3", torch.float8_e5m2: "e5m2"}


def mc2_quant_all_reduce(x_chunks: Sequence[torch.Tensor], scale_chunks: Sequence[torch.Tensor], *,
                         x_kind: Optional[str] = None, out_dtype: torch.dtype = torch.bfloat16,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """QuantAllReduce of the ranks' quantised shards resident on this GPU.

    x_chunks: world_size tensors (bs, h) or (b, s, h) of one-byte codes: int8,
    float8_e4m3fn or float8_e5m2 (or uint8 with ``x_kind`` "int8" | "e4m3" |
    "e5m2").  scale_chunks: fp32 (bs, h/128) per-token-per-group scales, or e8m0
    codes (bs, h/64, 2) as uint8 (mx).  Returns out of the same leading shape
    as x in ``out_dtype`` (fp32, fp16 or bf16).
    """
    if stream is not None:
        return _on_stream(mc2_quant_all_reduce, locals())
    cur = _current_device()
    x0 = x_chunks[0]
    if x_kind is None:
        if x0.dtype not in _QAR_X_BY_DTYPE:
            raise ValueError("x_kind is required for x of dtype %s" % x0.dtype)
        x_kind = _QAR_X_BY_DTYPE[x0.dtype]
    h = x0.shape[-1]
    bs = x0.numel() // h
    if len(scale_chunks) != len(x_chunks):
        raise ValueError(f"scale_chunks must hold {len(x_chunks)} tensors (one per rank), got {len(scale_chunks)}")
    xp = _args(x_chunks, x0.shape, x0.dtype, "x_chunks", cur)
    s0 = scale_chunks[0]
    sdt = MC2_F32 if s0.dtype == torch.float32 else MC2_E8M0
    # fp32: one scale per token per 128 elements, any shape; e8m0: one uint8 code per 32
    sdtype = torch.float32 if sdt == MC2_F32 else torch.uint8
    if h % 128 == 0:
        count = bs * (h // 128 if sdt == MC2_F32 else h // 32)
        for i, sc in enumerate(scale_chunks):
            if sc.numel() != count or sc.dtype != sdtype:
                raise ValueError(f"scale_chunks[{i}] must hold {count} "
                                 f"{'fp32 scales' if sdt == MC2_F32 else 'e8m0 codes (uint8)'}, "
                                 f"got {sc.numel()} of {sc.dtype}")
    sp = _args(scale_chunks, s0.shape, sdtype, "scale_chunks", cur)
    if out is None:
        out = torch.empty(x0.shape, dtype=out_dtype, device=x0.device)
    outp = _arg(out, x0.shape, out_dtype, "out", cur)
    _need_device(cur)
    st = lib().mc2_quant_all_reduce(xp, sp, len(x_chunks), bs, h, _QAR_X[x_kind], sdt, _dtype_code(out.dtype),
                                    outp, _stream(stream, cur))
    _check(st)
    return out


def mc2_alltoall_quant_mm_workspace(rank_size: int, bs_local: int, h: int, n: int, x1_quant_mode: int,
                                    x1_dtype: torch.dtype) -> int:
    nbytes = ctypes.c_size_t(0)
    _check(lib().mc2_alltoall_quant_mm_workspace(rank_size, bs_local, h, n, x1_quant_mode, _dtype_code(x1_dtype),
                                                 ctypes.byref(nbytes)))
    return int(nbytes.value)


def _a2a_args(chunks, x2, x2_scale, bias, x1_quant_mode, x1_scale, out, q_out, x1_scale_out, acc_out,
              alltoall_out, cur: int) -> list:
    """The pointers of an AlltoAllQuantMatmul call, each tensor checked against
    the sizes of the first chunk and of x2 (the quant modes and the 16-bit /
    int8 choice are the library's to refuse)."""
    R = len(chunks)
    bs_local, h = chunks[0].shape
    K = R * h
    n = x2.shape[1]
    x1_dtype = chunks[0].dtype
    if bias.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"bias must be of dtype torch.float32 or torch.bfloat16, got {bias.dtype}")
    if x1_quant_mode == QUANT_PERTOKEN:
        x1p = _opt(x1_scale, (bs_local,), torch.float32, "x1_scale (per-token scale)", cur)
    else:
        x1p = _opt(x1_scale, (K,), x1_dtype, "x1_scale (smooth scale)", cur)
    return [_args(chunks, (bs_local, h), x1_dtype, "chunks", cur), x1p,
            _arg(x2, (K, n), torch.int8, "x2", cur),
            _arg(x2_scale, (n,), torch.float32, "x2_scale", cur),
            _arg(bias, (n,), bias.dtype, "bias", cur),
            _arg(out, (bs_local, n), torch.bfloat16, "out", cur),
            _opt(alltoall_out, (R, bs_local, h), x1_dtype, "alltoall_out", cur),
            _opt(q_out, (bs_local, K), torch.int8, "q_out", cur),
            _opt(x1_scale_out, (bs_local,), torch.float32, "x1_scale_out", cur),
            _opt(acc_out, (bs_local, n), torch.int32, "acc_out", cur)]


def mc2_alltoall_quant_mm(chunks: Sequence[torch.Tensor], x2: torch.Tensor, x2_scale: torch.Tensor,
                          bias: torch.Tensor, *, x1_quant_mode: int, x1_scale: Optional[torch.Tensor] = None,
                          x2_quant_mode: int = QUANT_PERCHANNEL, out: Optional[torch.Tensor] = None,
                          q_out: Optional[torch.Tensor] = None, x1_scale_out: Optional[torch.Tensor] = None,
                          acc_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          alltoall_out: Optional[torch.Tensor] = None, stream=None) -> dict:
    """AlltoAllQuantMatmul on the received chunks already resident on this GPU.

    chunks: rank_size tensors (bs_local, h) (bf16/fp16 for mode 7, int8 for
    mode 3); x2 int8 (rank_size*h, n); x2_scale fp32 (n); bias fp32/bf16 (n).
    alltoall_out: optional (rank_size, bs_local, h) tensor of the chunks' dtype
    that receives commOut (the chunks stacked, before the permute).
    Returns dict(out, q, x1_scale, acc, alltoall_out) with the optional outputs
    that were given.
    """
    if stream is not None:
        return _on_stream(mc2_alltoall_quant_mm, locals())
    cur = _current_device()
    R = len(chunks)
    bs_local, h = chunks[0].shape
    n = x2.shape[1]
    dev = chunks[0].device
    x1_dtype = chunks[0].dtype
    if out is None:
        out = torch.empty((bs_local, n), dtype=torch.bfloat16, device=dev)
    a = _a2a_args(chunks, x2, x2_scale, bias, x1_quant_mode, x1_scale, out, q_out, x1_scale_out, acc_out,
                  alltoall_out, cur)
    _need_device(cur)
    if workspace is None:
        need = mc2_alltoall_quant_mm_workspace(R, bs_local, h, n, x1_quant_mode, x1_dtype)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wp = _arg(workspace, workspace.shape, workspace.dtype, "workspace", cur)
    st = lib().mc2_alltoall_quant_mm(a[0], R, bs_local, h, _dtype_code(x1_dtype), a[1], a[2], a[3], a[4],
                                     _dtype_code(bias.dtype), x1_quant_mode, x2_quant_mode, n, a[5], a[6], a[7],
                                     a[8], a[9], wp, workspace.numel() * workspace.element_size(),
                                     _stream(stream, cur))
    _check(st)
    return {"out": out, "q": q_out, "x1_scale": x1_scale_out, "acc": acc_out, "alltoall_out": alltoall_out}


NO_ALLOC_SCRATCH_BYTES = 32 << 20


def mc2_alltoall_quant_mm_no_alloc(chunks: Sequence[torch.Tensor], x2: torch.Tensor, x2_scale: torch.Tensor,
                                   bias: torch.Tensor, *, x1_quant_mode: int, out: torch.Tensor,
                                   x1_scale: Optional[torch.Tensor] = None, x2_quant_mode: int = QUANT_PERCHANNEL,
                                   q_out: Optional[torch.Tensor] = None, x1_scale_out: Optional[torch.Tensor] = None,
                                   acc_out: Optional[torch.Tensor] = None, alltoall_out: Optional[torch.Tensor] = None,
                                   stream=None) -> dict:
    """The same computation as mc2_alltoall_quant_mm without a workspace.

    For callers that cannot allocate device memory: the library's built-in
    scratch (NO_ALLOC_SCRATCH_BYTES per GPU) is used instead, so problems whose
    workspace would exceed it are refused.  ``out`` must be given (nothing is
    allocated here).  Calls that may overlap on the GPU share that scratch and
    must be serialised by the caller.
    """
    cur = _current_device()
    if out is None:
        raise ValueError("out must be given (this entry point allocates nothing)")
    R = len(chunks)
    bs_local, h = chunks[0].shape
    n = x2.shape[1]
    a = _a2a_args(chunks, x2, x2_scale, bias, x1_quant_mode, x1_scale, out, q_out, x1_scale_out, acc_out,
                  alltoall_out, cur)
    _need_device(cur)
    st = lib().mc2_alltoall_quant_mm_no_alloc(a[0], R, bs_local, h, _dtype_code(chunks[0].dtype), a[1], a[2], a[3],
                                              a[4], _dtype_code(bias.dtype), x1_quant_mode, x2_quant_mode, n, a[5],
                                              a[6], a[7], a[8], a[9], _stream(stream, cur))
    _check(st)
    return {"out": out, "q": q_out, "x1_scale": x1_scale_out, "acc": acc_out, "alltoall_out": alltoall_out}


# ------------------------------------------------------------------ around the linears
# These calls take matrices whose rows are strided (a slice of a wider tensor),
# and tensors of more dimensions, whose last one is the row: (b, s, h) is the
# (b * s, h) problem.

def _rows(t: torch.Tensor, shape, dtype, what: str, cur: int):
    """The tensor's device pointer and its row stride in elements, once its shape, dtype, device and
    layout are right: rows of adjacent elements at one stride."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != cur:
        _refuse(t, shape, dtype, what, cur)
    cols = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), cols
    ld = None
    ok = cols == 1 or t.stride(-1) == 1
    rows = 1                      # rows below the dimension looked at
    for d in range(t.dim() - 2, -1, -1):
        if shape[d] == 1:
            continue
        if ld is None:
            ld = t.stride(d)
        elif t.stride(d) != rows * ld:
            ok = False
        rows *= shape[d]
    if ld is None:
        ld = cols
    if not ok or ld < cols:
        raise ValueError(f"{what} must have rows of adjacent elements at one stride, got strides {t.stride()} "
                         f"for shape {tuple(shape)}")
    return t.data_ptr(), ld


def _opt_rows(t: Optional[torch.Tensor], shape, dtype, what: str, cur: int):
    return (None, 0) if t is None else _rows(t, shape, dtype, what, cur)


_contiguous = torch.contiguous_format


def _like(t: torch.Tensor) -> torch.Tensor:
    """A new contiguous tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=_contiguous)


def _leading(t: torch.Tensor, what: str) -> int:
    """The number of rows of a tensor of two or more dimensions."""
    if t.dim() == 2:
        return t.shape[0]
    if t.dim() < 2:
        raise ValueError(f"{what} must have at least 2 dimensions, got {t.dim()}")
    rows = 1
    for n in t.shape[:-1]:
        rows *= n
    return rows


_QNORM = {torch.int8: MC2_I8, torch.float8_e4m3fn: MC2_F8E4M3, torch.float8_e5m2: MC2_F8E5M2}


def mc2_add_rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, quant_mode: int = QUANT_NONE, q_dtype: torch.dtype = torch.int8,
                     with_out: Optional[bool] = None, with_rstd: bool = False, out: Optional[torch.Tensor] = None,
                     residual_out: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                     q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None) -> dict:
    """RMS norm of x + residual, with 8-bit codes for the fused linear that follows.

    x, residual (..., h) of fp16, bf16 or fp32; weight (h) of x's type or fp32.
    quant_mode: QUANT_NONE; QUANT_PERTOKEN_DYNAMIC (scale fp32, one per row: what
    mc2_alltoall_quant_mm takes in mode 3); QUANT_PERGROUP (fp32, one per 128
    columns) or QUANT_MX (e8m0 codes as uint8, one per 32 columns), the layouts of
    mc2_quant_all_reduce.  q_dtype: int8, float8_e4m3fn or float8_e5m2.  The 16-bit
    ``out`` is made when there are no codes, when it is given, or by ``with_out``.
    Returns dict(out, residual, rstd, q, scale): the sum that was normalised is
    ``residual`` (None without a residual); outputs not asked for are None.
    """
    if stream is not None:
        return _on_stream(mc2_add_rms_norm, locals())
    cur = _current_device()
    if cur >= 0:
        r = (_native_module or _native()).add_rms_norm(x, weight, residual, eps, quant_mode, q_dtype, with_out, with_rstd,
                                                       out, residual_out, rstd, q, scale, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    shape, dt, dev = x.shape, x.dtype, x.device
    m, h = _leading(x, "x"), shape[-1]
    xp, ldx = _rows(x, shape, dt, "x", cur)
    wt = weight.dtype
    wp = _arg(weight, (h,), wt, "weight", cur)
    rp, ldr = _opt_rows(residual, shape, dt, "residual", cur)
    op, ldo, rop, ldro = None, 0, None, 0
    if out is not None or with_out or (with_out is None and quant_mode == QUANT_NONE):
        if out is None: 
            out = torch.empty(shape, dtype=dt, device=dev)
            op, ldo = out.data_ptr(), h
        else:
            op, ldo = _rows(out, shape, dt, "out", cur)
    if residual_out is not None:
        rop, ldro = _rows(residual_out, shape, dt, "residual_out", cur)
    elif residual is not None:
        residual_out = _like(x)
        rop, ldro = residual_out.data_ptr(), h
    sp = None
    if rstd is not None or with_rstd:
        if rstd is None:
            rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        sp = _arg(rstd, shape[:-1], torch.float32, "rstd", cur)
    qp, scp, qd = None, None, 0
    if quant_mode != QUANT_NONE:
        if q_dtype not in _QNORM:
            raise ValueError(f"q_dtype must be int8, float8_e4m3fn or float8_e5m2, got {q_dtype}")
        qd = _QNORM[q_dtype]
        if q is None:
            q = torch.empty(shape, dtype=q_dtype, device=dev)
            qp = q.data_ptr()
        else:
            qp = _arg(q, shape, q_dtype, "q", cur)
        sshape, sdt = shape[:-1], torch.float32
        if quant_mode == QUANT_PERGROUP:
            sshape = (*sshape, -(-h // 128))
        elif quant_mode == QUANT_MX:
            sshape, sdt = (*sshape, -(-h // 32)), torch.uint8
        if scale is None:
            scale = torch.empty(sshape, dtype=sdt, device=dev)
            scp = scale.data_ptr()
        else:
            scp = _arg(scale, sshape, sdt, "scale", cur)
    elif q is not None or scale is not None:
        raise ValueError("q and scale need a quant_mode")
    _need_device(cur)
    _check(lib().mc2_add_rms_norm(xp, ldx, rp, ldr, wp, _dtype_code(wt), m, h, eps, _dtype_code(dt), op, ldo, rop,
                                  ldro, sp, quant_mode, qd, qp, scp, _stream(stream, cur)))
    return {"out": out if op is not None else None, "residual": residual_out, "rstd": rstd, "q": q, "scale": scale}


@functools.lru_cache(maxsize=1024)
def mc2_rms_norm_grad_workspace(m: int, h: int) -> int:
    nbytes = ctypes.c_size_t(0)
    _check(lib().mc2_rms_norm_grad_workspace(m, h, ctypes.byref(nbytes)))
    return int(nbytes.value)


def mc2_rms_norm_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                      dres: Optional[torch.Tensor] = None, with_weight: bool = True,
                      dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of mc2_add_rms_norm's ``out``.

    x is what was normalised (the forward call's ``residual`` output, or x itself
    without one) and rstd its ``rstd``; dres is the gradient that arrives at the
    ``residual`` output.  Returns (dx, dw): dx is the gradient of both x and the
    residual, dw of the weight (None without ``with_weight``).
    """
    if stream is not None:
        return _on_stream(mc2_rms_norm_grad, locals())
    cur = _current_device()
    if cur >= 0:
        r = (_native_module or _native()).rms_norm_grad(dy, x, weight, rstd, dres, with_weight, dx, dw, workspace, cur,
                                                        _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    shape, dt, dev = x.shape, x.dtype, x.device
    m, h = _leading(x, "x"), shape[-1]
    xp, ldx = _rows(x, shape, dt, "x", cur)
    dyp, lddy = _rows(dy, shape, dt, "dy", cur)
    wt = weight.dtype
    wp = _arg(weight, (h,), wt, "weight", cur)
    sp = _arg(rstd, shape[:-1], torch.float32, "rstd", cur)
    drp, lddr = _opt_rows(dres, shape, dt, "dres", cur)
    if dx is None:
        dx = _like(x)
        dxp, lddx = dx.data_ptr(), h
    else:
        dxp, lddx = _rows(dx, shape, dt, "dx", cur)
    dwp, wsp, nbytes = None, None, 0
    if with_weight or dw is not None:
        if dw is None:
            dw = _like(weight)
            dwp = dw.data_ptr()
        else:
            dwp = _arg(dw, (h,), wt, "dw", cur)
        _need_device(cur)
        if workspace is None:
            nbytes = mc2_rms_norm_grad_workspace(m, h)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            wsp = workspace.data_ptr()
        else:
            wsp = _arg(workspace, workspace.shape, workspace.dtype, "workspace", cur)
            nbytes = workspace.numel() * workspace.element_size()
    _need_device(cur)
    _check(lib().mc2_rms_norm_grad(dyp, lddy, xp, ldx, wp, _dtype_code(wt), sp, drp, lddr, m, h, _dtype_code(dt), dxp,
                                   lddx, dwp, wsp, nbytes, _stream(stream, cur)))
    return dx, dw


_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(name: str) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}, got {name!r}")
    return _ACTIVATIONS[name]


def mc2_matmul_bias_act(x: torch.Tensor, w: torch.Tensor, *, w_is_nk: bool = True,
                        bias: Optional[torch.Tensor] = None, activation: str = "none",
                        residual: Optional[torch.Tensor] = None, with_preact: bool = False,
                        out: Optional[torch.Tensor] = None, preact: Optional[torch.Tensor] = None, stream=None):
    """out = act(x @ w^T + bias) + residual, in one kernel.

    x (..., k); w (n, k), or (k, n) with ``w_is_nk=False``; bias (n); residual
    (..., n); all of one 16-bit type.  activation: "none", "relu", "gelu" (by erf),
    "gelu_tanh" or "silu".  Returns (out, preact): preact = x @ w^T + bias, with
    ``with_preact`` or when given, is what the gradients take.
    """
    if stream is not None:
        return _on_stream(mc2_matmul_bias_act, locals())
    cur = _current_device()
    act = _activation(activation)
    if cur >= 0:
        r = (_native_module or _native()).matmul_bias_act(x, w, w_is_nk, bias, act, residual, with_preact, out, preact,
                                                          cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    dt, dev = x.dtype, x.device
    m, k = _leading(x, "x"), x.shape[-1]
    if w.dim() != 2:
        raise ValueError(f"w must have 2 dimensions, got {w.dim()}")
    n = w.shape[0] if w_is_nk else w.shape[1]
    xp, ldx = _rows(x, x.shape, dt, "x", cur)
    wp, ldw = _rows(w, (n, k) if w_is_nk else (k, n), dt, "w", cur)
    bp = _opt(bias, (n,), dt, "bias", cur)
    oshape = (*x.shape[:-1], n)
    rp, ldr = _opt_rows(residual, oshape, dt, "residual", cur)
    if out is None:
        out = torch.empty(oshape, dtype=dt, device=dev)
        op, ldo = out.data_ptr(), n
    else:
        op, ldo = _rows(out, oshape, dt, "out", cur)
    pp, ldp = None, 0
    if preact is not None:
        pp, ldp = _rows(preact, oshape, dt, "preact", cur)
    elif with_preact:
        preact = torch.empty(oshape, dtype=dt, device=dev)
        pp, ldp = preact.data_ptr(), n
    _need_device(cur)
    _check(lib().mc2_matmul_bias_act(xp, ldx, wp, ldw, w_is_nk, m, n, k, bp, act, rp, ldr, _dtype_code(dt), op, ldo,
                                     pp, ldp, _stream(stream, cur)))
    return out, preact


def mc2_matmul_act_grad(dy: torch.Tensor, w: torch.Tensor, z: torch.Tensor, *, activation: str, w_is_nk: bool = True,
                        dz: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dz = (dy @ w) * act'(z): the gradient of z for y = act(z) @ w^T.

    dy (..., n); w (n, k), or (k, n) with ``w_is_nk=False``; z (..., k), the forward
    call's ``preact``.  The layer's dW and dB are mc2_matmul_weight_grad(dy, act(z)).
    """
    if stream is not None:
        return _on_stream(mc2_matmul_act_grad, locals())
    cur = _current_device()
    act = _activation(activation)
    if cur >= 0:
        r = (_native_module or _native()).matmul_act_grad(dy, w, z, act, w_is_nk, dz, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    dt = dy.dtype
    m, n = _leading(dy, "dy"), dy.shape[-1]
    if w.dim() != 2:
        raise ValueError(f"w must have 2 dimensions, got {w.dim()}")
    k = w.shape[1] if w_is_nk else w.shape[0]
    dyp, lddy = _rows(dy, dy.shape, dt, "dy", cur)
    wp, ldw = _rows(w, (n, k) if w_is_nk else (k, n), dt, "w", cur)
    zshape = (*dy.shape[:-1], k)
    zp, ldz = _rows(z, zshape, dt, "z", cur)
    if dz is None:
        dz = torch.empty(zshape, dtype=dt, device=dy.device)
        dzp, lddz = dz.data_ptr(), k
    else:
        dzp, lddz = _rows(dz, zshape, dt, "dz", cur)
    _need_device(cur)
    _check(lib().mc2_matmul_act_grad(dyp, lddy, wp, ldw, w_is_nk, zp, ldz, act, m, n, k, _dtype_code(dt), dzp, lddz,
                                     _stream(stream, cur)))
    return dz


def mc2_act_grad(dy: torch.Tensor, z: torch.Tensor, *, activation: str, dz: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """dz = dy * act'(z), elementwise: the gradient of mc2_matmul_bias_act's
    ``preact`` for a gradient ``dy`` of its ``out``."""
    if stream is not None:
        return _on_stream(mc2_act_grad, locals())
    cur = _current_device()
    act = _activation(activation)
    if cur >= 0:
        r = (_native_module or _native()).act_grad(dy, z, act, dz, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    shape, dt = dy.shape, dy.dtype
    m = _leading(dy, "dy")
    dyp, lddy = _rows(dy, shape, dt, "dy", cur)
    zp, ldz = _rows(z, shape, dt, "z", cur)
    if dz is None:
        dz = torch.empty(shape, dtype=dt, device=dy.device)
        dzp, lddz = dz.data_ptr(), shape[-1]
    else:
        dzp, lddz = _rows(dz, shape, dt, "dz", cur)
    _need_device(cur)
    _check(lib().mc2_act_grad(dyp, lddy, zp, ldz, act, m, shape[-1], _dtype_code(dt), dzp, lddz,
                              _stream(stream, cur)))
    return dz


# ------------------------------------------------------------------ the 8-bit path of a linear

def _kept(q: torch.Tensor, scale: torch.Tensor, cur: int):
    """The pointers, quant mode and code type of codes (..., h) and their scales, whose type and shape say
    what they are scales of: fp32 (...) of rows, fp32 (..., ceil(h / 128)) or uint8 (..., ceil(h / 32)) of groups."""
    if q.dtype not in _QNORM:
        raise ValueError(f"q must be of dtype int8, float8_e4m3fn or float8_e5m2, got {q.dtype}")
    _leading(q, "q")
    shape, h = q.shape[:-1], q.shape[-1]
    sdt, mode = torch.float32, QUANT_PERTOKEN_DYNAMIC
    if scale.dtype == torch.uint8:
        shape, sdt, mode = (*shape, -(-h // 32)), torch.uint8, QUANT_MX
    elif scale.dim() == q.dim():
        shape, mode = (*shape, -(-h // 128)), QUANT_PERGROUP
    return _arg(q, q.shape, q.dtype, "q", cur), _arg(scale, shape, sdt, "scale", cur), mode, _QNORM[q.dtype]


def _workspace(given: Optional[torch.Tensor], nbytes: int, device, cur: int):
    """A workspace's tensor, pointer and size: the one given, or one of nbytes."""
    if given is None:
        given = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return given, _arg(given, given.shape, given.dtype, "workspace", cur), given.numel() * given.element_size()


def mc2_quant_matmul(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
                     w_is_nk: bool = True, bias: Optional[torch.Tensor] = None, activation: str = "none",
                     residual: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """out = act((x @ w^T) * x_scale * w_scale + bias) + residual: int8 codes, exact integer sums.

    x (..., k) int8 with x_scale (...) fp32, one per row (mc2_add_rms_norm's or mc2_act_quant's codes and scales with
    QUANT_PERTOKEN_DYNAMIC); w (n, k) int8, or (k, n) with ``w_is_nk=False``, with w_scale (n) fp32; bias (n) of the
    output's type or fp32; residual (..., n).  dtype: the output's, float16 or bfloat16 (by default out's or residual's,
    else bfloat16).  k is at most 131071.  ``workspace``, if given, holds mc2_quant_matmul_workspace(...) bytes.
    """
    if stream is not None:
        return _on_stream(mc2_quant_matmul, locals())
    cur = _current_device()
    act = _activation(activation)
    dt = dtype if dtype is not None else out.dtype if out is not None else residual.dtype if residual is not None else torch.bfloat16
    if cur >= 0:
        r = (_native_module or _native()).quant_matmul(x, x_scale, w, w_scale, w_is_nk, bias, act, residual, dt, out, workspace,
                                                       cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    m, k = _leading(x, "x"), x.shape[-1]
    if w.dim() != 2:
        raise ValueError(f"w must have 2 dimensions, got {w.dim()}")
    n = w.shape[0] if w_is_nk else w.shape[1]
    xp, ldx = _rows(x, x.shape, torch.int8, "x", cur)
    xsp = _arg(x_scale, x.shape[:-1], torch.float32, "x_scale", cur)
    wp, ldw = _rows(w, (n, k) if w_is_nk else (k, n), torch.int8, "w", cur)
    wsp = _arg(w_scale, (n,), torch.float32, "w_scale", cur)
    bp, bdt = None, dt
    if bias is not None:
        bdt = torch.float32 if bias.dtype == torch.float32 else dt
        bp = _arg(bias, (n,), bdt, "bias", cur)
    oshape = (*x.shape[:-1], n)
    rp, ldr = _opt_rows(residual, oshape, dt, "residual", cur)
    _dtype_code(dt)
    if out is None:
        out = torch.empty(oshape, dtype=dt, device=x.device)
        op, ldo = out.data_ptr(), n
    else:
        op, ldo = _rows(out, oshape, dt, "out", cur)
    _need_device(cur)
    nbytes = ctypes.c_size_t(0)
    if workspace is None:
        _check(lib().mc2_quant_matmul_workspace(xp, ldx, wp, ldw, w_is_nk, m, n, k, rp, ldr, op, ldo,
                                                ctypes.byref(nbytes)))
    workspace, ws, size = _workspace(workspace, nbytes.value, x.device, cur)
    _check(lib().mc2_quant_matmul(xp, ldx, xsp, wp, ldw, w_is_nk, wsp, m, n, k, bp, _dtype_code(bdt), act, rp, ldr, _dtype_code(dt),
                                  op, ldo, ws, size, _stream(stream, cur)))
    return out


def mc2_quant_matmul_workspace(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor, *, w_is_nk: bool = True,
                               residual: Optional[torch.Tensor] = None) -> int:
    """Bytes of workspace that mc2_quant_matmul needs for these matrices."""
    cur = _current_device()
    m, k = _leading(x, "x"), x.shape[-1]
    n = w.shape[0] if w_is_nk else w.shape[1]
    xp, ldx = _rows(x, x.shape, torch.int8, "x", cur)
    wp, ldw = _rows(w, (n, k) if w_is_nk else (k, n), torch.int8, "w", cur)
    op, ldo = _rows(out, (*x.shape[:-1], n), out.dtype, "out", cur)
    rp, ldr = _opt_rows(residual, (*x.shape[:-1], n), out.dtype, "residual", cur)
    nbytes = ctypes.c_size_t(0)
    _check(lib().mc2_quant_matmul_workspace(xp, ldx, wp, ldw, w_is_nk, m, n, k, rp, ldr, op, ldo, ctypes.byref(nbytes)))
    return int(nbytes.value)


def mc2_act_quant(z: torch.Tensor, *, activation: str = "none", quant_mode: int = QUANT_PERTOKEN_DYNAMIC,
                  q_dtype: torch.dtype = torch.int8, q: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, stream=None):
    """The 8-bit codes of act(z) and their scales: (q, scale).

    z (..., h) of fp16, bf16 or fp32.  quant_mode and q_dtype, and the scales they give, as in mc2_add_rms_norm:
    QUANT_PERTOKEN_DYNAMIC, QUANT_PERGROUP or QUANT_MX; int8, float8_e4m3fn or float8_e5m2.  Without an activation z
    itself is kept in 8 bits (for mc2_act_grad_quant and mc2_matmul_weight_grad_quant); with one, the codes
    are the next linear's input (int8 per token: mc2_quant_matmul's x).
    """
    if stream is not None:
        return _on_stream(mc2_act_quant, locals())
    cur = _current_device()
    act = _activation(activation)
    if cur >= 0:
        r = (_native_module or _native()).act_quant(z, act, quant_mode, q_dtype, q, scale, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    shape, dev = z.shape, z.device
    m, h = _leading(z, "z"), shape[-1]
    zp, ldz = _rows(z, shape, z.dtype, "z", cur)
    if q_dtype not in _QNORM:
        raise ValueError(f"q_dtype must be int8, float8_e4m3fn or float8_e5m2, got {q_dtype}")
    sshape, sdt = shape[:-1], torch.float32
    if quant_mode == QUANT_PERGROUP:
        sshape = (*sshape, -(-h // 128))
    elif quant_mode == QUANT_MX:
        sshape, sdt = (*sshape, -(-h // 32)), torch.uint8
    if q is None:
        q = torch.empty(shape, dtype=q_dtype, device=dev)
    qp = _arg(q, shape, q_dtype, "q", cur)
    if scale is None:
        scale = torch.empty(sshape, dtype=sdt, device=dev)
    sp = _arg(scale, sshape, sdt, "scale", cur)
    _need_device(cur)
    _check(lib().mc2_act_quant(zp, ldz, m, h, act, _dtype_code(z.dtype), quant_mode, _QNORM[q_dtype], qp, sp, _stream(stream, cur)))
    return q, scale


def mc2_act_dequant(q: torch.Tensor, scale: torch.Tensor, *, activation: str = "none", dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(q * scale), rounded once to ``dtype`` (float16, bfloat16 or float32; by default out's, else bfloat16).

    q (..., h) int8, float8_e4m3fn or float8_e5m2; scale as mc2_act_quant and mc2_add_rms_norm make it: fp32 (...) per
    token, fp32 (..., ceil(h / 128)) per 128 columns or uint8 (..., ceil(h / 32)) e8m0 codes.
    """
    if stream is not None:
        return _on_stream(mc2_act_dequant, locals())
    cur = _current_device()
    act = _activation(activation)
    dt = dtype if dtype is not None else out.dtype if out is not None else torch.bfloat16
    if cur >= 0:
        r = (_native_module or _native()).act_dequant(q, scale, act, dt, out, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    qp, sp, mode, qd = _kept(q, scale, cur)
    m, h = _leading(q, "q"), q.shape[-1]
    _dtype_code(dt)
    if out is None:
        out = torch.empty(q.shape, dtype=dt, device=q.device)
        op, ldo = out.data_ptr(), h
    else:
        op, ldo = _rows(out, q.shape, dt, "out", cur)
    _need_device(cur)
    _check(lib().mc2_act_dequant(qp, sp, m, h, act, mode, qd, _dtype_code(dt), op, ldo, _stream(stream, cur)))
    return out


def mc2_act_grad_quant(dy: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *, activation: str,
                       dz: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dz = dy * act'(q * scale), elementwise: mc2_act_grad for a pre-activation kept in 8 bits (``dz`` may be dy)."""
    if stream is not None:
        return _on_stream(mc2_act_grad_quant, locals())
    cur = _current_device()
    act = _activation(activation)
    if cur >= 0:
        r = (_native_module or _native()).act_grad_quant(dy, q, scale, act, dz, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    qp, sp, mode, qd = _kept(q, scale, cur)
    shape, dt = q.shape, dy.dtype
    m, h = _leading(q, "q"), shape[-1]
    dyp, lddy = _rows(dy, shape, dt, "dy", cur)
    if dz is None:
        dz = torch.empty(shape, dtype=dt, device=dy.device)
        dzp, lddz = dz.data_ptr(), h
    else:
        dzp, lddz = _rows(dz, shape, dt, "dz", cur)
    _need_device(cur)
    _check(lib().mc2_act_grad_quant(dyp, lddy, qp, sp, m, h, act, mode, qd, _dtype_code(dt), dzp, lddz, _stream(stream, cur)))
    return dz


def mc2_matmul_weight_grad_quant(dy: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *, activation: str = "none",
                                 with_bias: bool = True, dw: Optional[torch.Tensor] = None,
                                 db: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """dw = dy^T @ act(q * scale) (n, k) and, with ``with_bias``, db = dy.sum(0) (n): (dw, db).

    mc2_matmul_weight_grad for an input kept in 8 bits: dy (..., n) of float16 or bfloat16, q (..., k) with its scales as
    in mc2_act_dequant.  With an activation, q is the pre-activation that the linear's input came from.
    ``workspace``, if given, holds mc2_matmul_weight_grad_quant_workspace(...) bytes.
    """
    if stream is not None:
        return _on_stream(mc2_matmul_weight_grad_quant, locals())
    cur = _current_device()
    act = _activation(activation)
    if cur >= 0:
        r = (_native_module or _native()).weight_grad_quant(dy, q, scale, act, with_bias, dw, db, workspace, cur, _stream(stream, cur))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    qp, sp, mode, qd = _kept(q, scale, cur)
    m, k, dt = _leading(q, "q"), q.shape[-1], dy.dtype
    _leading(dy, "dy")
    n = dy.shape[-1]
    dyp, lddy = _rows(dy, (*q.shape[:-1], n), dt, "dy", cur)
    if dw is None:
        dw = torch.empty((n, k), dtype=dt, device=dy.device)
    dwp = _arg(dw, (n, k), dt, "dw", cur)
    dbp = None
    if with_bias or db is not None:
        if db is None:
            db = torch.empty((n,), dtype=dt, device=dy.device)
        dbp = _arg(db, (n,), dt, "db", cur)
    _need_device(cur)
    nbytes = ctypes.c_size_t(0)
    if workspace is None:
        _check(lib().mc2_matmul_weight_grad_quant_workspace(dyp, lddy, dwp, m, n, k, ctypes.byref(nbytes)))
    workspace, ws, size = _workspace(workspace, nbytes.value, dy.device, cur)
    _check(lib().mc2_matmul_weight_grad_quant(dyp, lddy, qp, sp, m, n, k, act, mode, qd, _dtype_code(dt), dwp, dbp, ws, size,
                                              _stream(stream, cur)))
    return dw, db


def mc2_matmul_weight_grad_quant_workspace(dy: torch.Tensor, k: int, *, dw: Optional[torch.Tensor] = None) -> int:
    """Bytes of workspace that mc2_matmul_weight_grad_quant needs for this dy (..., n) and k columns of codes.

    For a ``dw`` of one's own that may not be 16-byte aligned, that too."""
    cur = _current_device()
    m, n = _leading(dy, "dy"), dy.shape[-1]
    dyp, lddy = _rows(dy, dy.shape, dy.dtype, "dy", cur)
    dwp = 16 if dw is None else _arg(dw, (n, k), dy.dtype, "dw", cur)
    nbytes = ctypes.c_size_t(0)
    _check(lib().mc2_matmul_weight_grad_quant_workspace(dyp, lddy, dwp, m, n, k, ctypes.byref(nbytes)))
    return int(nbytes.value)


def mc2_device_status() -> int:
    """Synchronise and return (and clear) the kernels' bounded-wait status."""
    return int(lib().mc2_device_status())


def mc2_set_launch_events(events: Optional[Sequence["torch.cuda.Event"]]) -> None:
    """Record the given CUDA events around the kernel launches of the next calls
    on this host thread: events[0] before a call's first launch, events[i]
    after its i-th (see the header for each call's launches).  None or [] turns
    it off.  The events must be created with timing enabled and stay alive
    while set."""
    evs = list(events or [])
    handles = [e.cuda_event for e in evs]
    if any(h == 0 for h in handles):
        raise ValueError("record each event once (or create it) before installing it")
    arr = (ctypes.c_void_p * max(1, len(handles)))(*handles) if handles else None
    _check(lib().mc2_set_launch_events(arr, len(handles)))


def mc2_test_expire_next_flag_waits(wait_limit_ns: int) -> None:
    """Test hook: the next AlltoAllQuantMatmul call on this host thread runs its
    GEMM with every stream-K finishing wait set to run out after
    ``wait_limit_ns`` (see the header)."""
    _check(lib().mc2_test_expire_next_flag_waits(int(wait_limit_ns)))


__all__ = [
    "Mc2Error", "lib", "library_path", "status_str", "last_error", "mc2_all_gather_mm",
    "mc2_matmul_reduce_scatter", "mc2_matmul_weight_grad", "mc2_quant_all_reduce",
    "mc2_alltoall_quant_mm_workspace", "mc2_alltoall_quant_mm",
    "mc2_alltoall_quant_mm_no_alloc",
    "mc2_add_rms_norm", "mc2_rms_norm_grad_workspace", "mc2_rms_norm_grad", "mc2_matmul_bias_act",
    "mc2_matmul_act_grad", "mc2_act_grad",
    "mc2_quant_matmul_workspace", "mc2_quant_matmul", "mc2_act_quant", "mc2_act_dequant", "mc2_act_grad_quant",
    "mc2_matmul_weight_grad_quant_workspace", "mc2_matmul_weight_grad_quant",
    "NO_ALLOC_SCRATCH_BYTES", "mc2_device_status", "mc2_set_launch_events", "mc2_test_expire_next_flag_waits",
    "MC2_OK", "MC2_ERR_NULL", "MC2_ERR_SHAPE", "MC2_ERR_DTYPE", "MC2_ERR_UNSUPPORTED", "MC2_ERR_WORKSPACE",
    "MC2_ERR_CUDA", "MC2_ERR_TIMEOUT", "MC2_F16", "MC2_BF16", "MC2_F32", "MC2_I8",
    "MC2_F8E4M3", "MC2_F8E5M2", "MC2_E8M0",
    "QUANT_NONE", "QUANT_PERCHANNEL", "QUANT_PERTOKEN", "QUANT_PERGROUP", "QUANT_MX", "QUANT_PERTOKEN_DYNAMIC",
]
