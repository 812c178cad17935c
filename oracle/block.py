"""fp64 CPU reference of the recurrent block's operators: the short causal convolution, the
selective state-space scan and the residual RMS norm, each with its gradients.

Plain loops over tokens, sequence by sequence, straight from the definitions; numpy only.
Test infrastructure: the library never calls it.
"""
from __future__ import annotations

import numpy as np


def sequences(B, T, cu=None):
    """(batch row, first row, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]


def _sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


# ------------------------------------------------------------ short convolution
def short_conv(x, w, bias=None, state=None, cu=None, silu=True):
    """x [B, T, C], w [C, W], state [N, W-1, C]: (y [B, T, C], final state); rows outside every
    sequence are zero."""
    B, T, C = x.shape
    W = w.shape[1]
    seqs = sequences(B, T, cu)
    y, end = np.zeros_like(x), np.zeros((len(seqs), W - 1, C))
    for n, (b, s, e) in enumerate(seqs):
        ext = np.concatenate([np.zeros((W - 1, C)) if state is None else state[n], x[b, s:e]])
        end[n] = ext[e - s:]
        for t in range(e - s):
            pre = (ext[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            y[b, s + t] = pre * _sigmoid(pre) if silu else pre
    return y, end


def short_conv_grads(x, w, dy, bias=None, state=None, dend=None, cu=None, silu=True):
    B, T, C = x.shape
    W = w.shape[1]
    seqs = sequences(B, T, cu)
    g = dict(dx=np.zeros_like(x), dw=np.zeros_like(w), db=np.zeros(C), ds=np.zeros((len(seqs), W - 1, C)))
    for n, (b, s, e) in enumerate(seqs):
        ext = np.concatenate([np.zeros((W - 1, C)) if state is None else state[n], x[b, s:e]])
        dext = np.zeros_like(ext)
        if dend is not None:
            dext[e - s:] += dend[n]
        for t in range(e - s):
            pre = (ext[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            sg = _sigmoid(pre)
            dp = dy[b, s + t] * (sg * (1 + pre * (1 - sg)) if silu else 1.0)
            g["dw"] += (dp * ext[t:t + W]).T
            g["db"] += dp
            dext[t:t + W] += dp * w.T
        g["ds"][n], g["dx"][b, s:e] = dext[:W - 1], dext[W - 1:]
    return g


# ------------------------------------------------------------------------- scan
def step_sizes(dt, dt_bias, softplus):
    v = dt + (0 if dt_bias is None else dt_bias)
    return np.logaddexp(0, v) if softplus else v


def ssm_scan(x, dt, A_log, Bm, Cm, D=None, dt_bias=None, h0=None, cu=None, softplus=True, keep=None):
    """x [B, T, H, P], dt [B, T, H], Bm, Cm [B, T, G, N], h0 [seqs, H, N, P]: (y, ht).  `keep`,
    a list, gets every (sequence, token)'s state before the token."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    seqs = sequences(B, T, cu)
    y, ht = np.zeros_like(x), np.zeros((len(seqs), H, N, P))
    d, of = step_sizes(dt, dt_bias, softplus), np.arange(H) // (H // G)
    dec = np.exp(-np.exp(A_log) * d)
    for n, (b, s, e) in enumerate(seqs):
        S = np.zeros((H, N, P)) if h0 is None else h0[n].copy()
        for t in range(s, e):
            if keep is not None:
                keep.append(S.copy())
            S = dec[b, t][:, None, None] * S + (d[b, t][:, None] * Bm[b, t, of])[:, :, None] * x[b, t][:, None]
            y[b, t] = np.einsum("hnp,hn->hp", S, Cm[b, t, of])
            if D is not None:
                y[b, t] += D[:, None] * x[b, t]
        ht[n] = S
    return y, ht


def ssm_scan_grads(x, dt, A_log, Bm, Cm, dy, D=None, dt_bias=None, h0=None, dht=None, cu=None,
                   softplus=True):
    """Reverse mode of the recurrence, token by token."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    seqs, before = sequences(B, T, cu), []
    ssm_scan(x, dt, A_log, Bm, Cm, D, dt_bias, h0, cu, softplus, keep=before)
    d, of, A = step_sizes(dt, dt_bias, softplus), np.arange(H) // (H // G), -np.exp(A_log)
    dec = np.exp(A * d)
    g = dict(dx=np.zeros_like(x), ddt=np.zeros_like(dt), dB=np.zeros_like(Bm), dC=np.zeros_like(Cm),
             dA_log=np.zeros(H), dD=np.zeros(H), ddt_bias=np.zeros(H), dh0=np.zeros((len(seqs), H, N, P)))
    at = sum(e - s for _, s, e in seqs)
    for n, (b, s, e) in reversed(list(enumerate(seqs))):
        E = np.zeros((H, N, P)) if dht is None else dht[n].copy()
        for t in reversed(range(s, e)):
            at -= 1
            old, bt, ct, xt, gt = before[at], Bm[b, t, of], Cm[b, t, of], x[b, t], dy[b, t]
            dd, dk = d[b, t], dec[b, t]
            S = dk[:, None, None] * old + (dd[:, None] * bt)[:, :, None] * xt[:, None]
            E = E + ct[:, :, None] * gt[:, None]
            for h in range(H):
                g["dC"][b, t, of[h]] += S[h] @ gt[h]
                g["dB"][b, t, of[h]] += dd[h] * (E[h] @ xt[h])
            g["dx"][b, t] = dd[:, None] * np.einsum("hnp,hn->hp", E, bt)
            if D is not None:
                g["dx"][b, t] += D[:, None] * gt
            g["dD"] += (gt * xt).sum(1)
            fade = dk * (E * old).sum((1, 2))         # through the decay's exponent
            ddt = np.einsum("hn,hnp,hp->h", bt, E, xt) + A * fade
            g["dA_log"] += fade * dd * A
            if softplus:
                ddt = ddt * _sigmoid(dt[b, t] + (0 if dt_bias is None else dt_bias))
            g["ddt"][b, t] = ddt
            g["ddt_bias"] += ddt
            E = dk[:, None, None] * E
        g["dh0"][n] = E
    return g


# ------------------------------------------------------------------------- norm
def add_rms_norm(x, w, res=None, eps=1e-6):
    h = x if res is None else x + res
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def add_rms_norm_grads(h, w, dy, eps=1e-6, dh=None):
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    xh, g = h * r, dy * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * xh).reshape(-1, h.shape[-1]).sum(0)


def round_e4m3(t):
    """The nearest 8-bit float (4 exponent bits, 3 fraction bits, top 448, ties to even)."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
    return np.clip(np.round(t / step) * step, -448, 448)


def quantise(y, kind, group):
    """(values in units of the scale, scale [rows, groups]) of y [rows, cols]."""
    top = 448.0 if kind == "e4m3" else 127.0
    cols = y.shape[1]
    size = group or cols
    q, scales = np.zeros_like(y), []
    for c in range(0, cols, size):
        part = y[:, c:c + size]
        m = np.abs(part).max(1, keepdims=True)
        s = np.where(m > 0, m / top, 1.0)
        t = part / s
        q[:, c:c + size] = round_e4m3(t) if kind == "e4m3" else np.round(t)
        scales.append(s)
    return q, np.concatenate(scales, 1)
