"""The gated delta rule with one decay per head and the norms around a gated block
(include/kda.h, "The gated delta rule with one decay per head" and "The norms around a gated
block").

Argument marshalling only, as in block.py: functions named as in C take preallocated tensors;
the others allocate their outputs, check their tensors and call them.  q, k and v, and the
gated norm's x and gate, may be column ranges of wider tensors (their rows are then read in
place); everything else is made contiguous.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _SIGNATURES, load
from .block import (_bad, _bytes, _code, _first_order, _indices, _nbytes, _no_grad, _offsets,
                    _on_device, _p, _rows, _s, _same_device, _want, _word)

__all__ = [
    "KDA_GDN_FLAG_QK_L2NORM", "KDA_GDN_FLAG_NO_SAVE", "KDA_GDN_FLAG_TEST_WAIT_TIMEOUT", "KDA_GATE_SIGMOID",
    "KDA_GATE_SILU",
    "KdaGdnShape", "KdaGatedNormShape", "KdaSandwichShape",
    "kda_gdn_fwd", "kda_gdn_bwd", "kda_gdn_workspace_size", "kda_gdn_bwd_workspace_size", "kda_gdn_step",
    "kda_gated_rmsnorm_fwd", "kda_gated_rmsnorm_bwd", "kda_gated_rmsnorm_bwd_workspace_size",
    "kda_sandwich_norm_fwd", "kda_sandwich_norm_bwd", "kda_sandwich_norm_bwd_workspace_size",
    "gated_delta_rule", "gated_delta_forward_save", "gated_delta_backward", "gated_delta_step",
    "gated_delta_autograd",
    "gated_rms_norm", "gated_rms_norm_backward", "gated_rms_norm_autograd",
    "sandwich_norm", "sandwich_norm_backward", "sandwich_norm_autograd",
]

KDA_GDN_FLAG_QK_L2NORM, KDA_GDN_FLAG_NO_SAVE, KDA_GDN_FLAG_TEST_WAIT_TIMEOUT = 1 << 0, 1 << 1, 1 << 31
KDA_GATE_SIGMOID, KDA_GATE_SILU = 0, 1


class KdaGdnShape(ctypes.Structure):
    """Mirror of `kda_gdn_shape` in include/kda.h."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("HV", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("g_scale", ctypes.c_float), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("flags", ctypes.c_uint32)]


class KdaGatedNormShape(ctypes.Structure):
    """Mirror of `kda_gated_norm_shape` in include/kda.h."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("group", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int), ("gate_first", ctypes.c_int32),
                ("shared_weight", ctypes.c_int32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64)]


class KdaSandwichShape(ctypes.Structure):
    """Mirror of `kda_sandwich_shape` in include/kda.h."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("eps", ctypes.c_float)]


_VP, _SZ, _I32, _ST = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int
_GDN, _GATED, _SAND = (ctypes.POINTER(s) for s in (KdaGdnShape, KdaGatedNormShape, KdaSandwichShape))
_SIGNATURES.update({
    "kda_gdn_fwd": (_ST, [_VP] * 7 + [_GDN] + [_VP] * 3 + [_SZ, _VP, _VP]),
    "kda_gdn_workspace_size": (_SZ, [_GDN]),
    "kda_gdn_bwd": (_ST, [_VP] * 7 + [_GDN] + [_VP] * 10 + [_SZ, _VP, _VP]),
    "kda_gdn_bwd_workspace_size": (_SZ, [_GDN, ctypes.c_int]),
    "kda_gdn_step": (_ST, [_VP] * 7 + [_I32, _GDN] + [_VP] * 3),
    "kda_gated_rmsnorm_fwd": (_ST, [_VP] * 3 + [_GATED] + [_VP] * 2),
    "kda_gated_rmsnorm_bwd": (_ST, [_VP] * 4 + [_GATED] + [_VP] * 4 + [_SZ, _VP]),
    "kda_gated_rmsnorm_bwd_workspace_size": (_SZ, [_GATED]),
    "kda_sandwich_norm_fwd": (_ST, [_VP] * 6 + [_SAND] + [_VP] * 3),
    "kda_sandwich_norm_bwd": (_ST, [_VP] * 8 + [_SAND] + [_VP] * 7 + [_SZ, _VP]),
    "kda_sandwich_norm_bwd_workspace_size": (_SZ, [_SAND]),
})


# ------------------------------------------------------------------ the C calls
def kda_gdn_fwd(q, k, v, g, beta, h0, cu_seqlens, shape: KdaGdnShape, o, ht, workspace, dev_status=None,
                stream=None):
    _check(load().kda_gdn_fwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(h0), _p(cu_seqlens),
                              ctypes.byref(shape), _p(o), _p(ht), _p(workspace), _nbytes(workspace),
                              _word(dev_status), _s(stream)))


def kda_gdn_workspace_size(shape: KdaGdnShape) -> int:
    return int(load().kda_gdn_workspace_size(ctypes.byref(shape)))


def kda_gdn_bwd(q, k, v, g, beta, h0, cu_seqlens, shape: KdaGdnShape, dout, dht, dq, dk, dv, dg, dbeta, dh0,
                saved, workspace, dev_status=None, stream=None):
    if saved is not None and _nbytes(saved, "saved") < kda_gdn_workspace_size(shape):
        _bad("saved is smaller than the forward's workspace for this shape")
    _check(load().kda_gdn_bwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(h0), _p(cu_seqlens),
                              ctypes.byref(shape), _p(dout), _p(dht), _p(dq), _p(dk), _p(dv), _p(dg),
                              _p(dbeta), _p(dh0), _p(saved), _p(workspace), _nbytes(workspace),
                              _word(dev_status), _s(stream)))


def kda_gdn_bwd_workspace_size(shape: KdaGdnShape, saved: bool) -> int:
    return int(load().kda_gdn_bwd_workspace_size(ctypes.byref(shape), int(bool(saved))))


def kda_gdn_step(q, k, v, g, beta, state, state_indices, num_slots: int, shape: KdaGdnShape, o,
                 dev_status=None, stream=None):
    _check(load().kda_gdn_step(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(state), _p(state_indices),
                               int(num_slots), ctypes.byref(shape), _p(o), _word(dev_status), _s(stream)))


def kda_gated_rmsnorm_fwd(x, gate, w, shape: KdaGatedNormShape, y, stream=None):
    _check(load().kda_gated_rmsnorm_fwd(_p(x), _p(gate), _p(w), ctypes.byref(shape), _p(y), _s(stream)))


def kda_gated_rmsnorm_bwd(dy, x, gate, w, shape: KdaGatedNormShape, dx, dgate, dw, workspace, stream=None):
    _check(load().kda_gated_rmsnorm_bwd(_p(dy), _p(x), _p(gate), _p(w), ctypes.byref(shape), _p(dx), _p(dgate),
                                        _p(dw), _p(workspace), _nbytes(workspace), _s(stream)))


def kda_gated_rmsnorm_bwd_workspace_size(shape: KdaGatedNormShape) -> int:
    return int(load().kda_gated_rmsnorm_bwd_workspace_size(ctypes.byref(shape)))


def kda_sandwich_norm_fwd(x, residual, gate, w_post, w_pre, residual_scale, shape: KdaSandwichShape, h, y,
                          stream=None):
    _check(load().kda_sandwich_norm_fwd(_p(x), _p(residual), _p(gate), _p(w_post), _p(w_pre),
                                        _p(residual_scale), ctypes.byref(shape), _p(h), _p(y), _s(stream)))


def kda_sandwich_norm_bwd(dy, dh, x, residual, gate, w_post, w_pre, residual_scale, shape: KdaSandwichShape,
                          dx, dresidual, dgate, dw_post, dw_pre, dresidual_scale, workspace, stream=None):
    _check(load().kda_sandwich_norm_bwd(_p(dy), _p(dh), _p(x), _p(residual), _p(gate), _p(w_post), _p(w_pre),
                                        _p(residual_scale), ctypes.byref(shape), _p(dx), _p(dresidual),
                                        _p(dgate), _p(dw_post), _p(dw_pre), _p(dresidual_scale),
                                        _p(workspace), _nbytes(workspace), _s(stream)))


def kda_sandwich_norm_bwd_workspace_size(shape: KdaSandwichShape) -> int:
    return int(load().kda_sandwich_norm_bwd_workspace_size(ctypes.byref(shape)))


# ------------------------------------------------------- the gated delta rule
def _gdn_setup(q, k, v, g, beta, initial_state, cu_seqlens, scale, g_scale, qk_l2norm, *more):
    _same_device(q, k, v, g, beta, initial_state, cu_seqlens, *more)
    if q.dim() != 4 or v.dim() != 4:
        _bad("q and k must be [B, T, H, K], v [B, T, HV, V]")
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    if k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        _bad(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}: expected [B, T, H, K] twice, "
             "[B, T, HV, V]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        _bad("k and v must have q's type")
    seqs = _offsets(cu_seqlens, B)
    g = _want("g", g, (B, T, HV), torch.float32)
    beta = _want("beta", beta, (B, T, HV), q.dtype)
    h0 = _want("initial_state", initial_state, (seqs, HV, K, V), torch.float32)
    (q, qs), (k, ks), (v, vs) = _rows(q, 2), _rows(k, 2), _rows(v, 2)
    shape = KdaGdnShape(B, T, H, HV, K, V, seqs, _code(q), _scale(scale), g_scale, qs, ks, vs,
                        KDA_GDN_FLAG_QK_L2NORM if qk_l2norm else 0)
    return (q, k, v, g, beta, h0, cu_seqlens), shape


def _scale(scale) -> float:
    if scale is None:
        return 0.0
    if not scale > 0:
        _bad(f"scale {scale} must be positive")
    return scale


def _gdn_forward(q, k, v, g, beta, scale, g_scale, qk_l2norm, initial_state, output_final_state, cu_seqlens,
                 workspace, dev_status, stream, save):
    _no_grad(q, k, v, g, beta, initial_state)
    ins, shape = _gdn_setup(q, k, v, g, beta, initial_state, cu_seqlens, scale, g_scale, qk_l2norm, workspace,
                            dev_status)
    if not save:
        shape.flags |= KDA_GDN_FLAG_NO_SAVE
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    ht = (torch.empty((shape.num_seqs, shape.HV, shape.K, shape.V), dtype=torch.float32, device=v.device)
          if output_final_state else None)
    if workspace is None:
        workspace = _bytes(kda_gdn_workspace_size(shape), v.device)
    kda_gdn_fwd(*ins, shape, o, ht, workspace, dev_status, stream)
    return o, ht, workspace


@_on_device
def gated_delta_forward_save(q, k, v, g, beta, *, scale=None, g_scale=1.0, qk_l2norm=False, initial_state=None,
                             output_final_state=False, cu_seqlens=None, workspace=None, dev_status=None,
                             stream=None):
    """gated_delta_rule that also returns its workspace, which holds each chunk's state and
    corrected values: (o, ht or None, saved).  gated_delta_backward(..., saved=saved) of the same
    inputs then does not form them again."""
    return _gdn_forward(q, k, v, g, beta, scale, g_scale, qk_l2norm, initial_state, output_final_state,
                        cu_seqlens, workspace, dev_status, stream, True)


@_on_device
def gated_delta_rule(q, k, v, g, beta, *, scale=None, g_scale=1.0, qk_l2norm=False, initial_state=None,
                     output_final_state=False, cu_seqlens=None, workspace=None, dev_status=None, stream=None):
    """The gated delta rule with one decay per head, chunked: q and k [B, T, H, K], v [B, T, HV, V]
    and beta [B, T, HV] (one type), g [B, T, HV] fp32 base-2 log decays (times g_scale: 1/ln 2 for
    natural ones); returns (o [B, T, HV, V], ht or None).  `initial_state` and ht are [N_seqs, HV,
    K, V] fp32; `scale` defaults to K^-1/2; `qk_l2norm` normalises q's and k's rows inside."""
    return _gdn_forward(q, k, v, g, beta, scale, g_scale, qk_l2norm, initial_state, output_final_state,
                        cu_seqlens, workspace, dev_status, stream, False)[:2]


@_on_device
def gated_delta_backward(q, k, v, g, beta, do, *, scale=None, g_scale=1.0, qk_l2norm=False, initial_state=None,
                         dht=None, cu_seqlens=None, saved=None, workspace=None, dev_status=None, stream=None):
    """The gradients of gated_delta_rule for do (and the final state's gradient dht): a dict of dq,
    dk, dv, dbeta in the inputs' type, dg and dinitial_state in fp32 (None without an initial
    state).  `saved`: gated_delta_forward_save's, for the same inputs."""
    ins, shape = _gdn_setup(*[None if t is None else t.detach() for t in (q, k, v, g, beta, initial_state)],
                            cu_seqlens, scale, g_scale, qk_l2norm, do, dht, saved, workspace, dev_status)
    do = _want("do", do.detach(), v.shape, v.dtype)
    dht = _want("dht", dht, (shape.num_seqs, shape.HV, shape.K, shape.V), torch.float32)
    if workspace is None:
        workspace = _bytes(kda_gdn_bwd_workspace_size(shape, saved is not None), q.device)
    out = {name: torch.empty(t.shape, dtype=t.dtype, device=t.device)
           for name, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    out["dinitial_state"] = None if initial_state is None else torch.empty_like(ins[5])
    kda_gdn_bwd(*ins, shape, do, dht, out["dq"], out["dk"], out["dv"], out["dg"], out["dbeta"],
                out["dinitial_state"], saved, workspace, dev_status, stream)
    return out


@_on_device
def gated_delta_step(q, k, v, g, beta, state, *, scale=None, g_scale=1.0, qk_l2norm=False, state_indices=None,
                     dev_status=None, stream=None):
    """One token per row: q and k [N, H, K], v [N, HV, V], g and beta [N, HV]; the cache `state`
    [slots, HV, K, V] fp32 is advanced in place at state_indices (int32 [N]; None: slot n;
    negative: an unused row, zero output).  Returns o [N, HV, V]."""
    _no_grad(q, k, v, g, beta, state)
    _same_device(q, k, v, g, beta, state, state_indices, dev_status)
    if q.dim() != 3 or v.dim() != 3:
        _bad("q and k must be [N, H, K], v [N, HV, V]")
    R, H, K = q.shape
    HV, V = v.shape[1:]
    if k.shape != q.shape or v.shape[0] != R:
        _bad(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}: expected [N, H, K] twice, [N, HV, V]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        _bad("k and v must have q's type")
    o = torch.empty((R, HV, V), dtype=q.dtype, device=q.device)
    if R == 0:
        return o
    if (not state.is_contiguous() or state.dtype != torch.float32 or state.dim() != 4
            or tuple(state.shape[1:]) != (HV, K, V)):
        _bad(f"state must be a contiguous fp32 [slots, {HV}, {K}, {V}] tensor (it is updated in place)")
    _indices(state_indices, R, state.shape[0])
    g = _want("g", g, (R, HV), torch.float32)
    beta = _want("beta", beta, (R, HV), q.dtype)
    (q, qs), (k, ks), (v, vs) = _rows(q, 1), _rows(k, 1), _rows(v, 1)
    shape = KdaGdnShape(R, 1, H, HV, K, V, R, _code(q), _scale(scale), g_scale, qs, ks, vs,
                        KDA_GDN_FLAG_QK_L2NORM if qk_l2norm else 0)
    kda_gdn_step(q, k, v, g, beta, state, state_indices, state.shape[0], shape, o, dev_status, stream)
    return o


class _GdnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, cu, scale, g_scale, qk_l2norm, save, dev_status):
        d = [None if t is None else t.detach() for t in (q, k, v, g, beta, h0)]
        ctx.kw = dict(scale=scale, g_scale=g_scale, qk_l2norm=qk_l2norm, dev_status=dev_status)
        kw = dict(initial_state=d[5], output_final_state=True, cu_seqlens=cu, **ctx.kw)
        saved = None
        if save:
            o, ht, saved = gated_delta_forward_save(*d[:5], **kw)
        else:
            o, ht = gated_delta_rule(*d[:5], **kw)
        ctx.save_for_backward(q, k, v, g, beta, h0, cu, saved)
        return o, ht

    @staticmethod
    @_first_order
    def backward(ctx, do, dht):
        q, k, v, g, beta, h0, cu, saved = ctx.saved_tensors
        d = gated_delta_backward(q, k, v, g, beta, do, initial_state=h0, dht=dht, cu_seqlens=cu, saved=saved,
                                 **ctx.kw)
        return (d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d["dinitial_state"], None, None, None, None,
                None, None)


def gated_delta_autograd(q, k, v, g, beta, *, scale=None, g_scale=1.0, qk_l2norm=False, initial_state=None,
                         cu_seqlens=None, save_for_backward=True, dev_status=None):
    """gated_delta_rule behind torch.autograd: (o, ht), with (first-order) gradients to every
    floating input.  With `save_for_backward` the chunk states are kept from the forward to the
    backward (kda_gdn_workspace_size bytes); False forms them again.  `dev_status` is given to the
    forward and to the backward."""
    return _GdnFunction.apply(q, k, v, g, beta, initial_state, cu_seqlens, scale, float(g_scale), bool(qk_l2norm),
                              bool(save_for_backward), dev_status)


# ------------------------------------------------------------------ gates
_GATES = {"sigmoid": KDA_GATE_SIGMOID, "silu": KDA_GATE_SILU}


def _act(name) -> int:
    if name not in _GATES:
        _bad(f"activation {name!r} (supported: 'sigmoid', 'silu')")
    return _GATES[name]


# ------------------------------------------------------------------ the gated norm
def _gated_setup(x, gate, weight, group, activation, gate_first, eps, *more):
    _same_device(x, gate, weight, *more)
    if x.dim() < 1 or x.shape[-1] < 1:
        _bad("x must have at least one column")
    if gate.shape != x.shape or gate.dtype != x.dtype:
        _bad(f"gate {tuple(gate.shape)} {gate.dtype} must have x's shape {tuple(x.shape)} and type {x.dtype}")
    cols = x.shape[-1]
    group = cols if group is None else group
    if weight.dtype != torch.float32 or tuple(weight.shape) not in ((group,), (cols,)):
        _bad(f"weight must be fp32 [{group}] (shared by the groups) or [{cols}]")
    weight = weight if weight.is_contiguous() else weight.contiguous()
    lead = x.dim() - 1
    (x, xs), (gate, gs) = _rows(x, lead), _rows(gate, lead)
    shape = KdaGatedNormShape(x.numel() // cols, cols, group, _code(x), _act(activation), int(bool(gate_first)),
                              int(weight.shape[0] == group), eps, xs, gs)
    return x, gate, weight, shape


@_on_device
def gated_rms_norm(x, gate, weight, *, group=None, activation="silu", gate_first=False, eps=1e-6, stream=None):
    """rms(x) weight act(gate), or with `gate_first` rms(x act(gate)) weight, over groups of `group`
    columns of the last dimension (None: all of them), rms(x) = x / sqrt(mean(x^2) + eps) and act
    'silu' or 'sigmoid'.  weight: fp32 [group], the same for every group, or [columns]."""
    _no_grad(x, gate, weight)
    x, gate, weight, shape = _gated_setup(x, gate, weight, group, activation, gate_first, eps)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    kda_gated_rmsnorm_fwd(x, gate, weight, shape, y, stream)
    return y


@_on_device
def gated_rms_norm_backward(dy, x, gate, weight, *, group=None, activation="silu", gate_first=False, eps=1e-6,
                            workspace=None, stream=None):
    """The gradients of gated_rms_norm for dy: a dict of dx, dgate (x's type) and dweight (fp32)."""
    x, gate, weight, shape = _gated_setup(x.detach(), gate.detach(), weight.detach(), group, activation, gate_first,
                                          eps, dy, workspace)
    dy = _want("dy", dy.detach(), x.shape, x.dtype)
    dx, dgate = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for _ in range(2))
    dw = torch.empty_like(weight)
    if workspace is None:
        workspace = _bytes(kda_gated_rmsnorm_bwd_workspace_size(shape), x.device)
    kda_gated_rmsnorm_bwd(dy, x, gate, weight, shape, dx, dgate, dw, workspace, stream)
    return {"dx": dx, "dgate": dgate, "dweight": dw}


class _GatedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight, group, activation, gate_first, eps):
        ctx.kw = dict(group=group, activation=activation, gate_first=gate_first, eps=eps)
        ctx.save_for_backward(x, gate, weight)
        return gated_rms_norm(x.detach(), gate.detach(), weight.detach(), **ctx.kw)

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        g = gated_rms_norm_backward(dy, *ctx.saved_tensors, **ctx.kw)
        return g["dx"], g["dgate"], g["dweight"], None, None, None, None


def gated_rms_norm_autograd(x, gate, weight, *, group=None, activation="silu", gate_first=False, eps=1e-6):
    """gated_rms_norm behind torch.autograd, with (first-order) gradients to x, gate and weight."""
    return _GatedFunction.apply(x, gate, weight, group, activation, bool(gate_first), eps)


# ------------------------------------------------------------------ the sandwich norm
def _sandwich_setup(x, residual, weight_post, weight_pre, gate, residual_scale, gate_activation, eps, *more):
    _same_device(x, residual, weight_post, weight_pre, gate, residual_scale, *more)
    if x.dim() < 1 or x.shape[-1] < 1:
        _bad("x must have at least one column")
    if gate is None and gate_activation is not None:
        _bad(f"gate_activation {gate_activation!r} without a gate")
    cols = x.shape[-1]
    x = x.contiguous()
    residual = _want("residual", residual, x.shape, x.dtype)
    gate = _want("gate", gate, x.shape, x.dtype)
    weight_post = _want("weight_post", weight_post, (cols,), torch.float32)
    weight_pre = _want("weight_pre", weight_pre, (cols,), torch.float32)
    residual_scale = _want("residual_scale", residual_scale, (cols,), torch.float32)
    act = KDA_GATE_SIGMOID if gate is None else _act(gate_activation)
    return ((x, residual, gate, weight_post, weight_pre, residual_scale),
            KdaSandwichShape(x.numel() // cols, cols, _code(x), act, eps))


@_on_device
def sandwich_norm(x, residual, weight_post, weight_pre, *, gate=None, gate_activation=None, residual_scale=None,
                  eps=1e-6, stream=None):
    """What stands between a block's output x and the next block's input: the residual stream
    h = residual_scale residual + act(gate) rms(x) weight_post and y = rms(h) weight_pre, over the
    last dimension; returns (y, h) in x's type.  gate (x's shape, with gate_activation 'silu' or
    'sigmoid') and residual_scale (fp32 [columns]) may be left out."""
    _no_grad(x, residual, weight_post, weight_pre, gate, residual_scale)
    ins, shape = _sandwich_setup(x, residual, weight_post, weight_pre, gate, residual_scale, gate_activation, eps)
    y, h = torch.empty_like(ins[0]), torch.empty_like(ins[0])
    kda_sandwich_norm_fwd(*ins, shape, h, y, stream)
    return y, h


@_on_device
def sandwich_norm_backward(dy, x, residual, weight_post, weight_pre, *, dresidual_out=None, gate=None,
                           gate_activation=None, residual_scale=None, eps=1e-6, workspace=None, stream=None):
    """The gradients of sandwich_norm for dy and the residual stream's own gradient dresidual_out (or
    None): a dict of dx, dresidual, dgate (x's type), dweight_post, dweight_pre and dresidual_scale
    (fp32); None for inputs not given."""
    ins, shape = _sandwich_setup(*[None if t is None else t.detach() for t in (
        x, residual, weight_post, weight_pre, gate, residual_scale)], gate_activation, eps, dy, dresidual_out,
        workspace)
    dy = _want("dy", dy.detach(), x.shape, x.dtype)
    dh = _want("dresidual_out", dresidual_out, x.shape, x.dtype)
    out = {"dx": torch.empty_like(ins[0]), "dresidual": torch.empty_like(ins[0]),
           "dgate": None if gate is None else torch.empty_like(ins[0]),
           "dweight_post": torch.empty_like(ins[3]), "dweight_pre": torch.empty_like(ins[4]),
           "dresidual_scale": None if residual_scale is None else torch.empty_like(ins[5])}
    if workspace is None:
        workspace = _bytes(kda_sandwich_norm_bwd_workspace_size(shape), x.device)
    kda_sandwich_norm_bwd(dy, dh, *ins, shape, *out.values(), workspace, stream)
    return out


class _SandwichFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight_post, weight_pre, gate, residual_scale, gate_activation, eps):
        ctx.kw = dict(gate_activation=gate_activation, eps=eps)
        ctx.save_for_backward(x, residual, weight_post, weight_pre, gate, residual_scale)
        d = [None if t is None else t.detach() for t in (x, residual, weight_post, weight_pre, gate, residual_scale)]
        return sandwich_norm(*d[:4], gate=d[4], residual_scale=d[5], **ctx.kw)

    @staticmethod
    @_first_order
    def backward(ctx, dy, dh):
        x, residual, weight_post, weight_pre, gate, residual_scale = ctx.saved_tensors
        g = sandwich_norm_backward(dy, x, residual, weight_post, weight_pre, dresidual_out=dh, gate=gate,
                                   residual_scale=residual_scale, **ctx.kw)
        return (g["dx"], g["dresidual"], g["dweight_post"], g["dweight_pre"], g["dgate"], g["dresidual_scale"],
                None, None)


def sandwich_norm_autograd(x, residual, weight_post, weight_pre, *, gate=None, gate_activation=None,
                           residual_scale=None, eps=1e-6):
    """sandwich_norm behind torch.autograd: (y, h), with (first-order) gradients to every tensor."""
    return _SandwichFunction.apply(x, residual, weight_post, weight_pre, gate, residual_scale, gate_activation, eps)
