"""The recurrent block's operators in fp64 torch, vectorised, for sizes at which the token loops of
oracle/block.py take too long: the formulas sequence by sequence, gradients by autograd."""
import torch
import torch.nn.functional as F


def spans(B, T, lens):
    """(batch row, first row, end) of every sequence."""
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    at, out = 0, []
    for n in lens:
        out.append((0, at, at + n))
        at += n
    return out


def conv(x, w, bias, state, lens, silu=True):
    """x [B, T, C], state [N, W-1, C] or None: (y, final states); rows outside every sequence are 0."""
    B, T, C = x.shape
    W, y, ends = w.shape[1], torch.zeros_like(x), []
    for n, (b, s, e) in enumerate(spans(B, T, lens)):
        ext = torch.cat([x.new_zeros(W - 1, C) if state is None else state[n], x[b, s:e]])
        pre = sum(ext[k:k + e - s] * w[:, k] for k in range(W)) + (0 if bias is None else bias)
        y = y.index_put((torch.tensor(b, device=x.device), torch.arange(s, e, device=x.device)),
                        pre * torch.sigmoid(pre) if silu else pre)
        ends.append(ext[e - s:])
    return y, torch.stack(ends)


def scan(x, dt, A_log, Bm, Cm, D, dt_bias, h0, lens, chunk=64):
    """x [B, T, H, P], dt [B, T, H], Bm, Cm [B, T, G, N], h0 [seqs, H, N, P]: (y, ht), in chunks
    whose decays are taken from differences of the running log decay."""
    B, T, H, P = x.shape
    per, ys, ends = H // Bm.shape[2], [torch.zeros_like(x[b]) for b in range(B)], []
    v = dt + dt_bias
    d = torch.where(v > 40, v, F.softplus(v, threshold=50.0))
    la = -torch.exp(A_log) * d
    for n, (b, s, e) in enumerate(spans(B, T, lens)):
        S, rows = h0[n], []
        for c in range(s, e, chunk):
            f = min(c + chunk, e)
            a = torch.cumsum(la[b, c:f], 0)                                   # [l, H]
            Bh, Ch = (t[b, c:f].repeat_interleave(per, 1) for t in (Bm, Cm))  # [l, H, N]
            xc, dc = x[b, c:f], d[b, c:f]
            gap = a[:, None] - a[None]                                        # [i, j, H]
            keep = torch.ones(f - c, f - c, dtype=torch.bool, device=x.device).tril()
            m = torch.exp(torch.where(keep[..., None], gap, -torch.inf)) * torch.einsum("ihn,jhn->ijh", Ch, Bh) * dc
            rows.append(torch.einsum("ijh,jhp->ihp", m, xc) + D[:, None] * xc
                        + torch.exp(a)[..., None] * torch.einsum("ihn,hnp->ihp", Ch, S))
            left = torch.exp(a[-1] - a) * dc
            S = torch.exp(a[-1])[:, None, None] * S + torch.einsum("jhn,jhp->hnp", Bh * left[..., None], xc)
        if rows:
            at = torch.arange(s, e, device=x.device)
            ys[b] = ys[b].index_put((at,), torch.cat(rows))
        ends.append(S)
    return torch.stack(ys), torch.stack(ends)


def norm(x, w, res=None, eps=1e-6):
    h = x if res is None else x + res
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w


def grads(f, inputs, douts):
    """d(sum of <output, dout>) / d(input) of the outputs f returns, for the inputs given (a dict)."""
    leaves = {k: v.detach().double().requires_grad_() for k, v in inputs.items() if v is not None}
    outs = f(**{k: leaves.get(k) for k in inputs})
    loss = sum((o * g.double()).sum() for o, g in zip(outs, douts) if g is not None)
    got = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return [o.detach() for o in outs], dict(zip(leaves, got))
