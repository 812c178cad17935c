"""The recurrent block's operators around KDA: the short causal convolution, the selective
state-space scan and the residual RMS norm (include/kda.h, "The recurrent block").

Argument marshalling only, as in the package's main module: functions named as in C take
preallocated tensors; the others allocate their outputs, check their tensors and call
them.  x, Bm and Cm of the scan and x of the convolution may be column ranges of a wider
tensor (their rows are then read in place); everything else is made contiguous.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import (KDA_DTYPE_BF16, KDA_DTYPE_F32, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KdaError,
               _check, _one_device, _SIGNATURES, load)

__all__ = [
    "KDA_CONV_FLAG_SILU", "KDA_SSM_FLAG_DT_SOFTPLUS", "KDA_SSM_FLAG_NO_SAVE", "KDA_NORM_SAME",
    "KDA_NORM_E4M3", "KDA_NORM_INT8", "KDA_DEVICE_BAD_INDEX", "KdaConvShape", "KdaSsmShape", "KdaNormShape",
    "kda_short_conv_fwd", "kda_short_conv_bwd", "kda_short_conv_bwd_workspace_size",
    "kda_short_conv_step", "kda_ssm_scan_fwd", "kda_ssm_scan_bwd", "kda_ssm_workspace_size",
    "kda_ssm_bwd_workspace_size", "kda_ssm_step", "kda_add_rmsnorm_fwd", "kda_add_rmsnorm_bwd",
    "kda_add_rmsnorm_bwd_workspace_size",
    "short_conv", "short_conv_backward", "short_conv_step", "short_conv_autograd",
    "ssm_scan", "ssm_scan_forward_save", "ssm_scan_backward", "ssm_step", "ssm_scan_autograd",
    "add_rms_norm", "add_rms_norm_quant", "add_rms_norm_backward", "add_rms_norm_autograd",
]

KDA_CONV_FLAG_SILU = 1 << 0
KDA_SSM_FLAG_DT_SOFTPLUS, KDA_SSM_FLAG_NO_SAVE = 1 << 0, 1 << 2
KDA_NORM_SAME, KDA_NORM_E4M3, KDA_NORM_INT8 = 0, 1, 2
KDA_DEVICE_BAD_INDEX = 1 << 4


class KdaConvShape(ctypes.Structure):
    """Mirror of `kda_conv_shape` in include/kda.h."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32),
                ("W", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("x_stride", ctypes.c_int64), ("flags", ctypes.c_uint32)]


class KdaSsmShape(ctypes.Structure):
    """Mirror of `kda_ssm_shape` in include/kda.h."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("G", ctypes.c_int32), ("N", ctypes.c_int32), ("P", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
                ("flags", ctypes.c_uint32)]


class KdaNormShape(ctypes.Structure):
    """Mirror of `kda_norm_shape` in include/kda.h."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("out", ctypes.c_int), ("group", ctypes.c_int32), ("eps", ctypes.c_float)]


_VP, _SZ, _I32, _ST = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int
_CONV, _SSM, _NORM = (ctypes.POINTER(s) for s in (KdaConvShape, KdaSsmShape, KdaNormShape))
_SIGNATURES.update({
    "kda_short_conv_fwd": (_ST, [_VP] * 5 + [_CONV] + [_VP] * 4),
    "kda_short_conv_bwd": (_ST, [_VP] * 5 + [_CONV] + [_VP] * 7 + [_SZ, _VP, _VP]),
    "kda_short_conv_bwd_workspace_size": (_SZ, [_CONV]),
    "kda_short_conv_step": (_ST, [_VP] * 5 + [_I32, _CONV] + [_VP] * 3),
    "kda_ssm_scan_fwd": (_ST, [_VP] * 9 + [_SSM] + [_VP] * 3 + [_SZ, _VP, _VP]),
    "kda_ssm_workspace_size": (_SZ, [_SSM]),
    "kda_ssm_scan_bwd": (_ST, [_VP] * 9 + [_SSM] + [_VP] * 12 + [_SZ, _VP, _VP]),
    "kda_ssm_bwd_workspace_size": (_SZ, [_SSM, ctypes.c_int]),
    "kda_ssm_step": (_ST, [_VP] * 9 + [_I32, _SSM] + [_VP] * 3),
    "kda_add_rmsnorm_fwd": (_ST, [_VP] * 3 + [_NORM] + [_VP] * 4),
    "kda_add_rmsnorm_bwd": (_ST, [_VP] * 4 + [_NORM] + [_VP] * 3 + [_SZ, _VP]),
    "kda_add_rmsnorm_bwd_workspace_size": (_SZ, [_NORM]),
})


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _s(stream):
    # the raw handle: current_stream() builds a Stream object, 3 us of a decode call
    return (torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None
            else stream.cuda_stream)


def _nbytes(t: Optional[torch.Tensor], name: str = "workspace") -> int:
    """The bytes that lie behind t's pointer."""
    if t is None:
        return 0
    if not t.is_contiguous():
        _bad(f"{name} must be contiguous: its size is counted in elements")
    return t.numel() * t.element_size()


def _word(t: Optional[torch.Tensor]):
    """dev_status, of which the kernels write the first four bytes."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() < 1:
        _bad("dev_status must be an int32 tensor of at least one element")
    return t.data_ptr()


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ the C calls
def kda_short_conv_fwd(x, w, bias, state_in, cu_seqlens, shape: KdaConvShape, y, state_out,
                       dev_status=None, stream=None):
    _check(load().kda_short_conv_fwd(_p(x), _p(w), _p(bias), _p(state_in), _p(cu_seqlens),
                                     ctypes.byref(shape), _p(y), _p(state_out), _word(dev_status),
                                     _s(stream)))


def kda_short_conv_bwd(x, w, bias, state_in, cu_seqlens, shape: KdaConvShape, dy, dstate_out, dx, dw,
                       dbias, dstate_in, workspace, dev_status=None, stream=None):
    _check(load().kda_short_conv_bwd(_p(x), _p(w), _p(bias), _p(state_in), _p(cu_seqlens),
                                     ctypes.byref(shape), _p(dy), _p(dstate_out), _p(dx), _p(dw),
                                     _p(dbias), _p(dstate_in), _p(workspace), _nbytes(workspace),
                                     _word(dev_status), _s(stream)))


def kda_short_conv_bwd_workspace_size(shape: KdaConvShape) -> int:
    return int(load().kda_short_conv_bwd_workspace_size(ctypes.byref(shape)))


def kda_short_conv_step(x, w, bias, state, state_indices, num_slots: int, shape: KdaConvShape, y,
                        dev_status=None, stream=None):
    _check(load().kda_short_conv_step(_p(x), _p(w), _p(bias), _p(state), _p(state_indices),
                                      int(num_slots), ctypes.byref(shape), _p(y), _word(dev_status),
                                      _s(stream)))


def kda_ssm_scan_fwd(x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu_seqlens, shape: KdaSsmShape, y, ht,
                     workspace, dev_status=None, stream=None):
    _check(load().kda_ssm_scan_fwd(_p(x), _p(dt), _p(A_log), _p(Bm), _p(Cm), _p(D), _p(dt_bias),
                                   _p(h0), _p(cu_seqlens), ctypes.byref(shape), _p(y), _p(ht),
                                   _p(workspace), _nbytes(workspace), _word(dev_status), _s(stream)))


def kda_ssm_workspace_size(shape: KdaSsmShape) -> int:
    return int(load().kda_ssm_workspace_size(ctypes.byref(shape)))


def kda_ssm_scan_bwd(x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu_seqlens, shape: KdaSsmShape, dy, dht,
                     dx, ddt, dB, dC, dA_log, dD, ddt_bias, dh0, saved, workspace, dev_status=None,
                     stream=None):
    if saved is not None and _nbytes(saved, "saved") < kda_ssm_workspace_size(shape):
        _bad("saved is smaller than the forward's workspace for this shape")
    _check(load().kda_ssm_scan_bwd(_p(x), _p(dt), _p(A_log), _p(Bm), _p(Cm), _p(D), _p(dt_bias),
                                   _p(h0), _p(cu_seqlens), ctypes.byref(shape), _p(dy), _p(dht),
                                   _p(dx), _p(ddt), _p(dB), _p(dC), _p(dA_log), _p(dD), _p(ddt_bias),
                                   _p(dh0), _p(saved), _p(workspace), _nbytes(workspace),
                                   _word(dev_status), _s(stream)))


def kda_ssm_bwd_workspace_size(shape: KdaSsmShape, saved: bool) -> int:
    return int(load().kda_ssm_bwd_workspace_size(ctypes.byref(shape), int(bool(saved))))


def kda_ssm_step(x, dt, A_log, Bm, Cm, D, dt_bias, state, state_indices, num_slots: int,
                 shape: KdaSsmShape, y, dev_status=None, stream=None):
    _check(load().kda_ssm_step(_p(x), _p(dt), _p(A_log), _p(Bm), _p(Cm), _p(D), _p(dt_bias),
                               _p(state), _p(state_indices), int(num_slots), ctypes.byref(shape),
                               _p(y), _word(dev_status), _s(stream)))


def kda_add_rmsnorm_fwd(x, residual, w, shape: KdaNormShape, h, y, scale, stream=None):
    _check(load().kda_add_rmsnorm_fwd(_p(x), _p(residual), _p(w), ctypes.byref(shape), _p(h), _p(y),
                                      _p(scale), _s(stream)))


def kda_add_rmsnorm_bwd(dy, h, w, dh, shape: KdaNormShape, dx, dw, workspace, stream=None):
    _check(load().kda_add_rmsnorm_bwd(_p(dy), _p(h), _p(w), _p(dh), ctypes.byref(shape), _p(dx),
                                      _p(dw), _p(workspace), _nbytes(workspace), _s(stream)))


def kda_add_rmsnorm_bwd_workspace_size(shape: KdaNormShape) -> int:
    return int(load().kda_add_rmsnorm_bwd_workspace_size(ctypes.byref(shape)))


# ------------------------------------------------------------------ checks
_DTYPES = {torch.bfloat16: KDA_DTYPE_BF16, torch.float32: KDA_DTYPE_F32}


def _bad(msg: str):
    raise KdaError(KDA_ERR_INVALID_ARG, msg)


def _code(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise KdaError(KDA_ERR_UNSUPPORTED, f"dtype {t.dtype} (supported: bfloat16, float32)")
    return code


def _want(name: str, t: Optional[torch.Tensor], shape, dtype) -> Optional[torch.Tensor]:
    """t, contiguous, or an error unless it has this shape and type (None passes)."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape):
        _bad(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        _bad(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t if t.is_contiguous() else t.contiguous()


def _rows(t: torch.Tensor, lead: int):
    """(tensor, elements between rows) of t viewed as [rows..., columns...] with `lead` row
    dimensions: t itself where the rows are evenly spaced and each row's columns are
    contiguous, else a contiguous copy (0: rows back to back)."""
    if t.is_contiguous():
        return t, 0
    size, stride = t.shape, t.stride()
    want, cols = 1, 1
    for d in range(t.dim() - 1, lead - 1, -1):
        if size[d] != 1 and stride[d] != want:
            return t.contiguous(), 0
        want *= size[d]
        cols *= size[d]
    step = span = None
    for d in range(lead - 1, -1, -1):
        if size[d] == 1:
            continue
        if step is None:
            step = stride[d]
            if step < cols:  # broadcast or overlapping rows
                return t.contiguous(), 0
            span = step * size[d]
        elif stride[d] != span:
            return t.contiguous(), 0
        else:
            span *= size[d]
    return (t.contiguous(), 0) if step is None else (t, step)  # None: one row


def _on_device(fn):
    """Run fn with its first argument's device current (the library launches there), and with
    `stream`, if given, as the current stream: outputs, workspaces and contiguous copies
    then belong to the stream whose kernels use them."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        first = args[0] if args else next((t for t in kwargs.values() if isinstance(t, torch.Tensor)), None)
        dev = -1 if first is None else first.get_device()
        if dev < 0:
            _bad("tensors must be on a CUDA device")
        stream = kwargs.get("stream")
        if stream is not None:
            with torch.cuda.stream(stream):
                return fn(*args, **kwargs)
        if dev == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(dev):
            return fn(*args, **kwargs)
    return wrapper


def _same_device(first, *ts):
    """Every given tensor on first's (CUDA) device, else KdaError."""
    dev = first.get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            _one_device(first, t)


def _no_grad(*ts):
    if not torch.is_grad_enabled():
        return
    for t in ts:
        if t is not None and t.requires_grad:
            raise KdaError(KDA_ERR_UNSUPPORTED,
                           "inputs requiring grad are rejected here: use the *_autograd functions")


def _offsets(cu: Optional[torch.Tensor], batch: int) -> int:
    """The number of sequences."""
    if cu is None:
        return batch
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 1 or not cu.is_contiguous():
        _bad("cu_seqlens must be a contiguous int32 vector of N + 1 offsets")
    return cu.numel() - 1


def _indices(idx: Optional[torch.Tensor], batch: int, slots: int):
    if idx is None:
        if slots < batch:
            _bad(f"{slots} state slots for {batch} rows without state_indices")
        return
    if idx.dtype != torch.int32 or tuple(idx.shape) != (batch,) or not idx.is_contiguous():
        _bad(f"state_indices must be a contiguous int32 vector of {batch} entries")


class _FirstOrder(torch.autograd.Function):
    """The last tensors given, as they are, behind a node that refuses to be differentiated."""
    @staticmethod
    def forward(ctx, made_from, *ts):
        return tuple(t.view_as(t) for t in ts[made_from:])

    @staticmethod
    def backward(ctx, *_):
        raise KdaError(KDA_ERR_UNSUPPORTED, "second-order gradients through the recurrent block's operators")


def _first_order(backward):
    """A backward whose gradients, asked for with create_graph=True, raise when they are
    differentiated: without a node between them and what they are made of they would pass for
    constants."""
    @functools.wraps(backward)
    def wrapper(ctx, *douts):
        with torch.no_grad():
            out = backward(ctx, *douts)
        if not torch.is_grad_enabled():
            return out
        of = [t for t in (*ctx.saved_tensors, *douts) if t is not None and t.requires_grad]
        kept = iter(_FirstOrder.apply(len(of), *of, *[g for g in out if g is not None]))
        return tuple(None if g is None else next(kept) for g in out)
    return wrapper


# ------------------------------------------------------- short convolution
def _conv_setup(x, weight, bias, initial_state, cu_seqlens, activation, *more):
    _same_device(x, weight, bias, initial_state, cu_seqlens, *more)
    if x.dim() != 3 or weight.dim() != 2:
        _bad("x must be [B, T, C] and weight [C, W]")
    if activation not in (None, "silu"):
        _bad(f"activation {activation!r} (supported: None, 'silu')")
    B, T, C = x.shape
    W = weight.shape[1]
    x, stride = _rows(x, 2)
    N = _offsets(cu_seqlens, B)
    shape = KdaConvShape(B, T, C, W, N, _code(x), stride, KDA_CONV_FLAG_SILU if activation else 0)
    weight = _want("weight", weight, (C, W), torch.float32)
    bias = _want("bias", bias, (C,), torch.float32)
    state = _want("initial_state", initial_state, (N, W - 1, C), x.dtype)
    return x, weight, bias, state, shape


@_on_device
def short_conv(x, weight, bias=None, *, initial_state=None, output_final_state=False,
               cu_seqlens=None, activation="silu", dev_status=None, stream=None):
    """The short causal depthwise convolution of x [B, T, C] with weight [C, W] and bias [C]
    (fp32), W in 2..4: returns (y [B, T, C], state or None).  `initial_state` and the
    returned state are [N, W-1, C]: the rows before, and the last rows of, each sequence."""
    _no_grad(x, weight, bias, initial_state)
    x, weight, bias, state, shape = _conv_setup(x, weight, bias, initial_state, cu_seqlens, activation,
                                                dev_status)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    out = (torch.empty((shape.num_seqs, shape.W - 1, shape.C), dtype=x.dtype, device=x.device)
           if output_final_state else None)
    kda_short_conv_fwd(x, weight, bias, state, cu_seqlens, shape, y, out, dev_status, stream)
    return y, out


@_on_device
def short_conv_backward(x, weight, dy, bias=None, *, initial_state=None, dfinal_state=None,
                        cu_seqlens=None, activation="silu", workspace=None, dev_status=None,
                        stream=None):
    """The gradients of short_conv for dy (and the final state's gradient): a dict of dx and
    dinitial_state (None without an initial state) in x's type, dweight and dbias (None
    without a bias) in fp32."""
    x, weight, bias, initial_state = [None if t is None else t.detach()
                                      for t in (x, weight, bias, initial_state)]
    x, weight, bias, state, shape = _conv_setup(x, weight, bias, initial_state, cu_seqlens, activation,
                                                dy, dfinal_state, dev_status, workspace)
    dy = _want("dy", dy.detach(), x.shape, x.dtype)
    dfinal = _want("dfinal_state", dfinal_state, (shape.num_seqs, shape.W - 1, shape.C), x.dtype)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    out = {"dx": dx, "dweight": torch.empty_like(weight),
           "dbias": None if bias is None else torch.empty_like(bias),
           "dinitial_state": None if state is None else torch.empty_like(state)}
    if workspace is None:
        workspace = _bytes(kda_short_conv_bwd_workspace_size(shape), x.device)
    kda_short_conv_bwd(x, weight, bias, state, cu_seqlens, shape, dy, dfinal, dx, out["dweight"],
                       out["dbias"], out["dinitial_state"], workspace, dev_status, stream)
    return out


@_on_device
def short_conv_step(x, state, weight, bias=None, *, state_indices=None, activation="silu",
                    dev_status=None, stream=None):
    """One token per row: x [N, C], the cache `state` [slots, W-1, C] moved on in place at
    state_indices (int32 [N]; None: slot n; negative: an unused row, zero output).  Returns
    y [N, C]."""
    _no_grad(x, state, weight, bias)
    _same_device(x, state, weight, bias, state_indices, dev_status)
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        _bad("x must be [N, C], weight [C, W] and state [slots, W-1, C]")
    if activation not in (None, "silu"):
        _bad(f"activation {activation!r} (supported: None, 'silu')")
    (N, C), W, slots = x.shape, weight.shape[1], state.shape[0]
    if N == 0:
        return torch.empty_like(x)
    _indices(state_indices, N, slots)
    if not state.is_contiguous() or state.dtype != x.dtype or tuple(state.shape[1:]) != (W - 1, C):
        _bad(f"state must be a contiguous [slots, {W - 1}, {C}] tensor of x's type (it is updated in place)")
    x, stride = _rows(x, 1)
    weight = _want("weight", weight, (C, W), torch.float32)
    bias = _want("bias", bias, (C,), torch.float32)
    y = torch.empty((N, C), dtype=x.dtype, device=x.device)
    shape = KdaConvShape(N, 1, C, W, N, _code(x), stride, KDA_CONV_FLAG_SILU if activation else 0)
    kda_short_conv_step(x, weight, bias, state, state_indices, slots, shape, y, dev_status, stream)
    return y


class _ConvFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, cu, activation, dev_status):
        d = [None if t is None else t.detach() for t in (x, weight, bias, state)]
        y, end = short_conv(d[0], d[1], d[2], initial_state=d[3], output_final_state=True,
                            cu_seqlens=cu, activation=activation, dev_status=dev_status)
        ctx.save_for_backward(x, weight, bias, state, cu)
        ctx.activation, ctx.dev_status = activation, dev_status
        return y, end

    @staticmethod
    @_first_order
    def backward(ctx, dy, dend):
        x, weight, bias, state, cu = ctx.saved_tensors
        g = short_conv_backward(x, weight, dy, bias, initial_state=state, dfinal_state=dend,
                                cu_seqlens=cu, activation=ctx.activation, dev_status=ctx.dev_status)
        return g["dx"], g["dweight"], g["dbias"], g["dinitial_state"], None, None, None


def short_conv_autograd(x, weight, bias=None, *, initial_state=None, cu_seqlens=None,
                        activation="silu", dev_status=None):
    """short_conv behind torch.autograd: (y, final state), with (first-order) gradients to x,
    weight, bias and the initial state.  `dev_status` is given to the forward and to the backward."""
    return _ConvFunction.apply(x, weight, bias, initial_state, cu_seqlens, activation, dev_status)


# ------------------------------------------------------------------ the scan
def _ssm_setup(x, dt, A_log, Bm, Cm, D, dt_bias, initial_state, cu_seqlens, dt_softplus, *more):
    _same_device(x, dt, A_log, Bm, Cm, D, dt_bias, initial_state, cu_seqlens, *more)
    if x.dim() != 4 or Bm.dim() != 4:
        _bad("x must be [B, T, H, P], Bm and Cm [B, T, G, N]")
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    if Bm.shape[:2] != x.shape[:2] or Cm.shape != Bm.shape or tuple(dt.shape) != (B, T, H):
        _bad(f"x {tuple(x.shape)}, dt {tuple(dt.shape)}, Bm {tuple(Bm.shape)}, Cm {tuple(Cm.shape)}: "
             "expected [B, T, H, P], [B, T, H], [B, T, G, N] twice")
    for name, t in (("dt", dt), ("Bm", Bm), ("Cm", Cm)):
        if t.dtype != x.dtype:
            _bad(f"{name} has dtype {t.dtype}, expected x's {x.dtype}")
    seqs = _offsets(cu_seqlens, B)
    A_log = _want("A_log", A_log, (H,), torch.float32)
    D = _want("D", D, (H,), torch.float32)
    dt_bias = _want("dt_bias", dt_bias, (H,), torch.float32)
    h0 = _want("initial_state", initial_state, (seqs, H, N, P), torch.float32)
    (x, xs), (dt, ds), (Bm, bs), (Cm, cs) = _rows(x, 2), _rows(dt, 2), _rows(Bm, 2), _rows(Cm, 2)
    shape = KdaSsmShape(B, T, H, G, N, P, seqs, _code(x), xs, ds, bs, cs,
                        KDA_SSM_FLAG_DT_SOFTPLUS if dt_softplus else 0)
    return (x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu_seqlens), shape


def _ssm_forward(x, dt, A_log, Bm, Cm, D, dt_bias, dt_softplus, initial_state, output_final_state,
                 cu_seqlens, workspace, dev_status, stream, save):
    _no_grad(x, dt, A_log, Bm, Cm, D, dt_bias, initial_state)
    ins, shape = _ssm_setup(x, dt, A_log, Bm, Cm, D, dt_bias, initial_state, cu_seqlens, dt_softplus,
                            workspace, dev_status)
    if not save:
        shape.flags |= KDA_SSM_FLAG_NO_SAVE
    dev = x.device
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    ht = (torch.empty((shape.num_seqs, shape.H, shape.N, shape.P), dtype=torch.float32, device=dev)
          if output_final_state else None)
    if workspace is None:
        workspace = _bytes(kda_ssm_workspace_size(shape), dev)
    kda_ssm_scan_fwd(*ins, shape, y, ht, workspace, dev_status, stream)
    return y, ht, workspace


@_on_device
def ssm_scan_forward_save(x, dt, A_log, Bm, Cm, *, D=None, dt_bias=None, dt_softplus=True,
                          initial_state=None, output_final_state=False, cu_seqlens=None,
                          workspace=None, dev_status=None, stream=None):
    """ssm_scan that also returns its workspace, which holds the state at each chunk's start:
    (y, ht or None, saved).  ssm_scan_backward(..., saved=saved) of the same inputs then does
    not form the states again."""
    return _ssm_forward(x, dt, A_log, Bm, Cm, D, dt_bias, dt_softplus, initial_state,
                        output_final_state, cu_seqlens, workspace, dev_status, stream, True)


@_on_device
def ssm_scan(x, dt, A_log, Bm, Cm, *, D=None, dt_bias=None, dt_softplus=True, initial_state=None,
             output_final_state=False, cu_seqlens=None, workspace=None, dev_status=None, stream=None):
    """The selective state-space scan of x [B, T, H, P] with steps dt [B, T, H], Bm and Cm
    [B, T, G, N] (one type), A_log, D and dt_bias [H] fp32; returns (y [B, T, H, P], ht or
    None).  `initial_state` and ht are [N_seqs, H, N, P] fp32."""
    return _ssm_forward(x, dt, A_log, Bm, Cm, D, dt_bias, dt_softplus, initial_state,
                        output_final_state, cu_seqlens, workspace, dev_status, stream, False)[:2]


@_on_device
def ssm_scan_backward(x, dt, A_log, Bm, Cm, dy, *, D=None, dt_bias=None, dt_softplus=True,
                      initial_state=None, dht=None, cu_seqlens=None, saved=None, workspace=None,
                      dev_status=None, stream=None):
    """The gradients of ssm_scan for dy (and the final state's gradient dht): a dict of dx,
    ddt, dB, dC in the inputs' type and dA_log, dD, ddt_bias, dh0 in fp32 (None for inputs
    not given).  `saved`: ssm_scan_forward_save's, for the same inputs."""
    ins, shape = _ssm_setup(*[None if t is None else t.detach()
                              for t in (x, dt, A_log, Bm, Cm, D, dt_bias, initial_state)],
                            cu_seqlens, dt_softplus, dy, dht, saved, workspace, dev_status)
    dy = _want("dy", dy.detach(), x.shape, x.dtype)
    dht = _want("dht", dht, (shape.num_seqs, shape.H, shape.N, shape.P), torch.float32)
    if workspace is None:
        workspace = _bytes(kda_ssm_bwd_workspace_size(shape, saved is not None), x.device)
    low = dict(dtype=x.dtype, device=x.device)
    out = {"dx": torch.empty(x.shape, **low), "ddt": torch.empty(dt.shape, **low),
           "dB": torch.empty(Bm.shape, **low), "dC": torch.empty(Cm.shape, **low),
           "dA_log": torch.empty_like(ins[2]),
           "dD": None if D is None else torch.empty_like(ins[5]),
           "ddt_bias": None if dt_bias is None else torch.empty_like(ins[6]),
           "dh0": None if initial_state is None else torch.empty_like(ins[7])}
    kda_ssm_scan_bwd(*ins, shape, dy, dht, out["dx"], out["ddt"], out["dB"], out["dC"], out["dA_log"],
                     out["dD"], out["ddt_bias"], out["dh0"], saved, workspace, dev_status, stream)
    return out


@_on_device
def ssm_step(x, dt, A_log, Bm, Cm, state, *, D=None, dt_bias=None, dt_softplus=True,
             state_indices=None, dev_status=None, stream=None):
    """One token per row: x [N, H, P], dt [N, H], Bm and Cm [N, G, Ns]; the cache `state`
    [slots, H, Ns, P] fp32 is advanced in place at state_indices (int32 [N]; None: slot n;
    negative: an unused row, zero output).  Returns y [N, H, P]."""
    _no_grad(x, dt, A_log, Bm, Cm, D, dt_bias, state)
    _same_device(x, dt, A_log, Bm, Cm, D, dt_bias, state, state_indices, dev_status)
    if x.dim() != 3 or Bm.dim() != 3 or state.dim() != 4:
        _bad("x must be [N, H, P], Bm and Cm [N, G, Ns], state [slots, H, Ns, P]")
    R, H, P = x.shape
    G, Ns = Bm.shape[1:]
    if Bm.shape[0] != R or Cm.shape != Bm.shape or tuple(dt.shape) != (R, H):
        _bad(f"x {tuple(x.shape)}, dt {tuple(dt.shape)}, Bm {tuple(Bm.shape)}, Cm {tuple(Cm.shape)}: "
             "expected [N, H, P], [N, H], [N, G, Ns] twice")
    if dt.dtype != x.dtype or Bm.dtype != x.dtype or Cm.dtype != x.dtype:
        _bad("dt, Bm and Cm must have x's type")
    if R == 0:
        return torch.empty_like(x)
    _indices(state_indices, R, state.shape[0])
    if not state.is_contiguous() or state.dtype != torch.float32 or tuple(state.shape[1:]) != (H, Ns, P):
        _bad(f"state must be a contiguous fp32 [slots, {H}, {Ns}, {P}] tensor (it is updated in place)")
    A_log = _want("A_log", A_log, (H,), torch.float32)
    D = _want("D", D, (H,), torch.float32)
    dt_bias = _want("dt_bias", dt_bias, (H,), torch.float32)
    (x, xs), (dt, ds), (Bm, bs), (Cm, cs) = _rows(x, 1), _rows(dt, 1), _rows(Bm, 1), _rows(Cm, 1)
    shape = KdaSsmShape(R, 1, H, G, Ns, P, R, _code(x), xs, ds, bs, cs,
                        KDA_SSM_FLAG_DT_SOFTPLUS if dt_softplus else 0)
    y = torch.empty((R, H, P), dtype=x.dtype, device=x.device)
    kda_ssm_step(x, dt, A_log, Bm, Cm, D, dt_bias, state, state_indices, state.shape[0], shape, y,
                 dev_status, stream)
    return y


class _SsmFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu, dt_softplus, save, dev_status):
        d = [None if t is None else t.detach() for t in (x, dt, A_log, Bm, Cm, D, dt_bias, h0)]
        kw = dict(D=d[5], dt_bias=d[6], dt_softplus=dt_softplus, initial_state=d[7],
                  output_final_state=True, cu_seqlens=cu, dev_status=dev_status)
        saved = None
        if save:
            y, ht, saved = ssm_scan_forward_save(*d[:5], **kw)
        else:
            y, ht = ssm_scan(*d[:5], **kw)
        ctx.dt_softplus, ctx.dev_status = dt_softplus, dev_status
        ctx.save_for_backward(x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu, saved)
        return y, ht

    @staticmethod
    @_first_order
    def backward(ctx, dy, dht):
        x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu, saved = ctx.saved_tensors
        g = ssm_scan_backward(x, dt, A_log, Bm, Cm, dy, D=D, dt_bias=dt_bias,
                              dt_softplus=ctx.dt_softplus, initial_state=h0, dht=dht, cu_seqlens=cu,
                              saved=saved, dev_status=ctx.dev_status)
        return (g["dx"], g["ddt"], g["dA_log"], g["dB"], g["dC"], g["dD"], g["ddt_bias"], g["dh0"],
                None, None, None, None)


def ssm_scan_autograd(x, dt, A_log, Bm, Cm, *, D=None, dt_bias=None, dt_softplus=True,
                      initial_state=None, cu_seqlens=None, save_for_backward=True, dev_status=None):
    """ssm_scan behind torch.autograd: (y, ht), with (first-order) gradients to every floating input.  With
    `save_for_backward` the chunk states are kept from the forward to the backward
    (kda_ssm_workspace_size bytes); False forms them again.  `dev_status` is given to the
    forward and to the backward."""
    return _SsmFunction.apply(x, dt, A_log, Bm, Cm, D, dt_bias, initial_state, cu_seqlens,
                              bool(dt_softplus), bool(save_for_backward), dev_status)


# ------------------------------------------------------------------ the norm
def _norm_setup(x, weight, eps, out=KDA_NORM_SAME, group=0):
    if x.dim() < 1 or x.shape[-1] < 1:
        _bad("x must have at least one column")
    cols = x.shape[-1]
    return KdaNormShape(x.numel() // cols, cols, _code(x), out, group, eps), _want("weight", weight, (cols,),
                                                                                  torch.float32)


@_on_device
def add_rms_norm(x, weight, *, residual=None, eps=1e-6, stream=None):
    """h = x + residual and y = h weight / sqrt(mean(h^2) + eps) over the last dimension:
    returns (y, h), both in x's type (h is x itself without a residual)."""
    _no_grad(x, weight, residual)
    _same_device(x, weight, residual)
    x = x.contiguous()
    shape, weight = _norm_setup(x, weight, eps)
    residual = _want("residual", residual, x.shape, x.dtype)
    y = torch.empty_like(x)
    h = x if residual is None else torch.empty_like(x)
    kda_add_rmsnorm_fwd(x, residual, weight, shape, None if residual is None else h, y, None, stream)
    return y, h


@_on_device
def add_rms_norm_quant(x, weight, *, residual=None, eps=1e-6, out_dtype="e4m3", group=0, stream=None):
    """add_rms_norm with an 8-bit output: returns (q, scale, h), q float8_e4m3fn or int8 of
    x's shape and scale [..., groups] fp32, one per row (group 0) or per 128 columns (group
    128): q * scale stands for the normalised row."""
    _no_grad(x, weight, residual)
    _same_device(x, weight, residual)
    kinds = {"e4m3": (KDA_NORM_E4M3, torch.float8_e4m3fn), "int8": (KDA_NORM_INT8, torch.int8)}
    if out_dtype not in kinds:
        _bad(f"out_dtype {out_dtype!r} (supported: 'e4m3', 'int8')")
    x = x.contiguous()
    code, dtype = kinds[out_dtype]
    shape, weight = _norm_setup(x, weight, eps, code, group)
    residual = _want("residual", residual, x.shape, x.dtype)
    q = torch.empty(x.shape, dtype=dtype, device=x.device)
    groups = -(-shape.cols // 128) if group else 1
    scale = torch.empty((*x.shape[:-1], groups), dtype=torch.float32, device=x.device)
    h = x if residual is None else torch.empty_like(x)
    kda_add_rmsnorm_fwd(x, residual, weight, shape, None if residual is None else h, q, scale, stream)
    return q, scale, h


@_on_device
def add_rms_norm_backward(dy, h, weight, *, eps=1e-6, dresidual=None, workspace=None, stream=None):
    """The gradients of add_rms_norm at its returned h, for dy and the residual stream's own
    gradient (or None): a dict of dx (x's and the residual's alike) and dweight (fp32)."""
    dy, h, weight = dy.detach(), h.detach().contiguous(), weight.detach()
    _same_device(dy, h, weight, dresidual, workspace)
    shape, weight = _norm_setup(h, weight, eps)
    dy = _want("dy", dy, h.shape, h.dtype)
    dresidual = _want("dresidual", dresidual, h.shape, h.dtype)
    dx, dw = torch.empty_like(h), torch.empty_like(weight)
    if workspace is None:
        workspace = _bytes(kda_add_rmsnorm_bwd_workspace_size(shape), h.device)
    kda_add_rmsnorm_bwd(dy, h, weight, dresidual, shape, dx, dw, workspace, stream)
    return {"dx": dx, "dweight": dw}


class _NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h = add_rms_norm(x.detach(), weight.detach(),
                            residual=None if residual is None else residual.detach(), eps=eps)
        ctx.save_for_backward(x if residual is None else h, weight)
        ctx.eps, ctx.has_res = eps, residual is not None
        return y, h.view_as(h) if residual is None else h

    @staticmethod
    @_first_order
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        g = add_rms_norm_backward(dy, h, weight, eps=ctx.eps, dresidual=dh)
        return g["dx"], g["dweight"], g["dx"] if ctx.has_res else None, None


def add_rms_norm_autograd(x, weight, *, residual=None, eps=1e-6):
    """add_rms_norm behind torch.autograd: (y, h), with (first-order) gradients to x, weight and
    residual."""
    return _NormFunction.apply(x, weight, residual, eps)
