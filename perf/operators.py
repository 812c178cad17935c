"""Cases of the recurrent block's operators: the short causal convolution, the selective
state-space scan and the residual RMS norm with an 8-bit output, for prompts, training
steps and single tokens.

With `own` false the operators run in plain form (elementary torch operations in fp32,
rounded once at the end); with `own` true they are the library's calls.

A case's "op" is one of
  conv        short causal convolution of a prompt (dense or packed), with SiLU and a state
  conv_train  its forward and its gradients
  conv_step   one new token for every sequence of a batch, state rows updated in place
  scan        selective state-space scan of a prompt (dense or packed), with final states
  scan_train  its forward and its gradients
  scan_step   one new token for every sequence, states updated in place
  norm        residual addition, RMS norm, output in 8 bits with scales
  norm_train  residual addition and RMS norm, and their gradients
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

LOG2E = 1.0 / math.log(2.0)
CHUNK = 64  # the plain scan's chunk length


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # the q, k, v projections of 16 heads x 128 channels of a training sequence, fused
        dict(name="conv_train_8k", op="conv_train", dtype="bf16", B=1, T=8192, C=6144, W=4, seqs=0,
             empty=0, lens_seed=0),
        # packed prompts in fp32 with carried state, an odd channel count
        dict(name="conv_packed_f32", op="conv", dtype="f32", B=1, T=15000, C=1537, W=3, seqs=24,
             empty=3, lens_seed=1),
        # decode: 512 sequences, one token each, rows of a larger state cache
        dict(name="conv_step_512", op="conv_step", dtype="bf16", N=512, C=6144, W=4),
        # a training sequence: 32 heads of 64, one group, as in a hybrid stack's layer
        dict(name="scan_train_8k", op="scan_train", dtype="bf16", B=1, T=8192, H=32, G=1, P=64,
             N=128, seqs=0, empty=0, lens_seed=0),
        # a long prompt of a wide layer
        dict(name="scan_prompt_8k", op="scan", dtype="bf16", B=1, T=8192, H=64, G=1, P=64, N=128,
             seqs=0, empty=0, lens_seed=0),
        # packed prompts with carried states, grouped B and C
        dict(name="scan_packed_12k", op="scan", dtype="bf16", B=1, T=12300, H=32, G=4, P=64, N=128,
             seqs=28, empty=3, lens_seed=3),
        # fp32 inputs, odd sizes everywhere
        dict(name="scan_f32_odd", op="scan", dtype="f32", B=2, T=777, H=6, G=2, P=40, N=24, seqs=0,
             empty=0, lens_seed=0),
        # decode: 512 sequences, one token each
        dict(name="scan_step_512", op="scan_step", dtype="bf16", N_seq=512, H=32, G=1, P=64, N=128),
        # decode of one sequence: latency
        dict(name="scan_step_1", op="scan_step", dtype="bf16", N_seq=1, H=32, G=1, P=64, N=128),
        # a prompt's block entry, the output in 8-bit floats for an 8-bit projection
        dict(name="norm_fp8_8k", op="norm", dtype="bf16", rows=8192, cols=4096, out="e4m3", group=128,
             residual=True),
        # one new token's block entry, 8-bit integers with one scale per token: latency
        dict(name="norm_int8_1", op="norm", dtype="bf16", rows=1, cols=4096, out="int8", group=0,
             residual=True),
        # a training step's block entry
        dict(name="norm_train_8k", op="norm_train", dtype="bf16", rows=8192, cols=2048, residual=True),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; 3072 is left out."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v - 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_train",
                     "scan_step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_step":
        return dict(op=op, dtype=dtype, N=_log(rng, 1, 512), C=_log(rng, 64, 6144),
                    W=rng.choice([2, 3, 4]))
    if op in ("conv", "conv_train"):
        packed = rng.random() < 0.5
        C = _log(rng, 64, 3000)
        C = C // 8 * 8 if rng.random() < 0.6 else C
        return dict(op=op, dtype=dtype, B=1 if packed else rng.choice([1, 2, 3]), T=_log(rng, 4, 5000),
                    C=C, W=rng.choice([2, 3, 4]), seqs=rng.randint(1, 20) if packed else 0,
                    empty=rng.randint(0, 3) if packed else 0, lens_seed=rng.randrange(1000))
    if op in ("scan", "scan_train", "scan_step"):
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4, 6, 8])
        P, N = rng.choice([(64, 128), (64, 128), (64, 64), (128, 64), (32, 16), (48, 80), (33, 20)])
        if H * P == 3072:
            H -= G
        if op == "scan_step":
            return dict(op=op, dtype=dtype, N_seq=_log(rng, 1, 400), H=H, G=G, P=P, N=N)
        packed = rng.random() < 0.5
        return dict(op=op, dtype=dtype, B=1 if packed else rng.choice([1, 2, 3]),
                    T=_log(rng, 2, 8192 if dtype == "bf16" else 2048), H=H, G=G, P=P, N=N,
                    seqs=rng.randint(1, 20) if packed else 0, empty=rng.randint(0, 3) if packed else 0,
                    lens_seed=rng.randrange(1000))
    cols = _log(rng, 64, 8192)
    cols = cols // 8 * 8 if rng.random() < 0.7 else cols
    case = dict(op=op, dtype=dtype, rows=_log(rng, 1, 8192), cols=cols, residual=rng.random() < 0.8)
    if op == "norm":
        case.update(out=rng.choice(["e4m3", "int8"]), group=rng.choice([0, 128]))
    return case


def _lens(case):
    """Sequence lengths of a case: equal when dense, else seeded cuts of [0, T] with empty
    slots among them (a cut may leave a sequence of one token)."""
    if not case["seqs"]:
        return [case["T"]] * case["B"]
    rng = random.Random(case["lens_seed"])
    n = min(case["seqs"], case["T"])
    cuts = sorted(rng.sample(range(1, case["T"]), n - 1)) if n > 1 else []
    lens = [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])] + [0] * case["empty"]
    rng.shuffle(lens)
    return lens


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ------------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev, dt, op = "cuda", _dt(case), case["op"]
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def rand(*shape, lo, hi):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = {"case": case}
    if op == "conv_step":
        N, C, W = case["N"], case["C"], case["W"]
        slots = N + N // 4 + 1
        s.update(x=randn(N, C), w=randn(C, W, std=W ** -0.5, dtype=torch.float32),
                 b=randn(C, std=0.1, dtype=torch.float32), state=randn(slots, W - 1, C),
                 idx=torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32))
    elif op in ("conv", "conv_train"):
        C, W, lens = case["C"], case["W"], _lens(case)
        s.update(x=randn(case["B"], case["T"], C), w=randn(C, W, std=W ** -0.5, dtype=torch.float32),
                 b=randn(C, std=0.1, dtype=torch.float32), state=randn(len(lens), W - 1, C))
        s["cu"] = _offsets(lens, dev) if case["seqs"] else None
        s["plan"] = _row_plan(lens, W, dev)
        if op == "conv_train":
            s["dy"] = randn(case["B"], case["T"], C)
    elif op in ("scan", "scan_train", "scan_step"):
        H, G, P, N = case["H"], case["G"], case["P"], case["N"]
        lens = _lens(case) if op != "scan_step" else []
        lead = (case["N_seq"],) if op == "scan_step" else (case["B"], case["T"])
        # x, B and C are column ranges of one convolved projection, as a layer has them
        s["xbc"] = randn(*lead, H * P + 2 * G * N)
        s["dt"] = randn(*lead, H)
        s["A_log"] = torch.log(rand(H, lo=1.0, hi=16.0))
        step = torch.exp(rand(H, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        s["D"] = 1.0 + randn(H, std=0.1, dtype=torch.float32)
        if op == "scan_step":
            slots = case["N_seq"] + case["N_seq"] // 4 + 1
            s["state"] = randn(slots, H, N, P, std=0.1, dtype=torch.float32)
            s["idx"] = torch.randperm(slots, generator=gen, device=dev)[:case["N_seq"]].to(torch.int32)
        else:
            s["h0"] = randn(len(lens), H, N, P, std=0.1, dtype=torch.float32)
            s["cu"] = _offsets(lens, dev) if case["seqs"] else None
            s["plan"] = _chunk_plan(lens, dev)
            if op == "scan_train":
                s["dy"] = randn(case["B"], case["T"], H, P)
    else:
        rows, cols = case["rows"], case["cols"]
        s.update(x=randn(rows, cols), w=1.0 + randn(cols, std=0.1, dtype=torch.float32),
                 res=randn(rows, cols, std=2.0) if case["residual"] else None)
        if op == "norm_train":
            s.update(dy=randn(rows, cols), dres=randn(rows, cols))
    return s


def _offsets(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)


def _row_plan(lens, W, dev):
    """For the plain convolution: the row each of a token's W taps reads in
    cat(tokens, state rows), and the row each final state entry reads."""
    n = torch.tensor(lens)
    seq = torch.repeat_interleave(torch.arange(len(lens)), n)
    start = torch.cumsum(n, 0) - n
    total = int(n.sum())
    at = torch.arange(total) - start[seq]
    src = (at[:, None] + torch.arange(W) - (W - 1))  # position within the sequence
    rows = torch.where(src >= 0, start[seq][:, None] + src, total + seq[:, None] * (W - 1) + src + W - 1)
    end = n[:, None] + torch.arange(W - 1) - (W - 1)
    ends = torch.where(end >= 0, start[:, None] + end,
                       total + torch.arange(len(lens))[:, None] * (W - 1) + end + W - 1)
    return {"rows": rows.to(dev), "ends": ends.to(dev)}


def _chunk_plan(lens, dev):
    """For the plain scan: every sequence padded to whole chunks; per padded row its token
    (or the zero row), per chunk its sequence, per sequence its first chunk and count."""
    n = torch.tensor(lens)
    nc = (n + CHUNK - 1) // CHUNK
    first = torch.cumsum(nc, 0) - nc
    start = torch.cumsum(n, 0) - n
    seq = torch.repeat_interleave(torch.arange(len(lens)), nc)
    at = (torch.arange(len(seq)) - first[seq])[:, None] * CHUNK + torch.arange(CHUNK)
    total = int(n.sum())
    row = torch.where(at < n[seq][:, None], start[seq][:, None] + at, total)
    back = torch.repeat_interleave((first * CHUNK - start), n) + torch.arange(total)
    return {"row": row.to(dev), "back": back.to(dev), "seq": seq.to(dev), "first": first.to(dev),
            "nc": nc.to(dev)}


# ------------------------------------------------------------------- plain forms
def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(x, w, b, state, plan):
    """x [rows, C], state [N, W-1, C] (fp32): y [rows, C] and the last W-1 rows of each sequence."""
    ext = torch.cat([x, state.flatten(0, 1)])
    rows = plan["rows"]
    pre = b + sum(ext[rows[:, k]] * w[:, k] for k in range(w.shape[1]))
    return _silu(pre), ext[plan["ends"]]


def _plain_dense_conv(x, w, b, state):
    """The same for equal sequences x [B, T, C], by shifted slices."""
    T, W = x.shape[1], w.shape[1]
    ext = torch.cat([state, x], 1)
    pre = b + sum(ext[:, k:k + T] * w[:, k] for k in range(W))
    return _silu(pre), ext[:, T:]


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20))))


def _plain_scan(x, dt, A_log, Bm, Cm, D, dt_bias, h0, plan):
    """The chunk form on padded chunks: x [rows, H, P], dt [rows, H], Bm, Cm [rows, G, N]
    (fp32); y [rows, H, P] and the final states [seqs, H, N, P]."""
    H, G = x.shape[1], Bm.shape[1]
    row, seq = plan["row"], plan["seq"]

    def chunks(t):  # [chunks, CHUNK, ...], zero rows past a sequence's end
        return torch.cat([t, torch.zeros_like(t[:1])])[row]

    d = chunks(_softplus(dt + dt_bias))                       # [c, l, H]
    a = torch.cumsum(d * -torch.exp(A_log), 1)                # log decay from the chunk's start
    xc, Bc, Cc = chunks(x), chunks(Bm), chunks(Cm)
    u = xc * d[..., None]
    l = torch.arange(CHUNK, device=x.device)
    gap = a[:, :, None] - a[:, None]                          # [c, i, j, H]
    gap = torch.where((l[:, None] >= l)[None, :, :, None], gap, -torch.inf)
    gram = torch.einsum("cign,cjgn->cijg", Cc, Bc).repeat_interleave(H // G, 3)
    y = torch.einsum("cijh,cjhp->cihp", gram * torch.exp(gap), u)
    left = torch.exp(a[:, -1:] - a)                           # decay to the chunk's end
    Bh = Bc.repeat_interleave(H // G, 2)
    local = torch.einsum("cjhn,cjhp->chnp", Bh, u * left[..., None])
    # the state at each chunk's start: every earlier chunk of its sequence, and h0, decayed
    run = torch.cat([torch.zeros_like(a[:1, -1]), torch.cumsum(a[:, -1], 0)])  # [c + 1, H]
    c = torch.arange(len(seq), device=x.device)
    same = (seq[:, None] == seq) & (c[:, None] > c)
    carry = torch.where(same[..., None], run[:-1, None] - run[None, 1:], -torch.inf)
    start = torch.einsum("cdh,dhnp->chnp", torch.exp(carry), local)
    start = start + torch.exp(run[:-1] - run[plan["first"][seq]])[..., None, None] * h0[seq]
    Ch = Cc.repeat_interleave(H // G, 2)
    y = y + torch.einsum("cihn,chnp->cihp", Ch, start) * torch.exp(a)[..., None]
    y = y + D[:, None] * xc
    some = plan["nc"] > 0
    last = torch.clamp(plan["first"] + plan["nc"] - 1, 0)
    last = torch.clamp(last, max=max(len(seq) - 1, 0))
    end = torch.exp(a[last, -1])[..., None, None] * start[last] + local[last]
    ht = torch.where(some[:, None, None, None], end, h0)
    return y.flatten(0, 1)[plan["back"]], ht


def _split(case, xbc):
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    x, Bm, Cm = xbc.split([H * P, G * N, G * N], -1)
    return x.unflatten(-1, (H, P)), Bm.unflatten(-1, (G, N)), Cm.unflatten(-1, (G, N))


def _plain_conv_step(s):
    idx = s["idx"].long()
    win = torch.cat([s["state"][idx].float(), s["x"].float()[:, None]], 1)  # [N, W, C]
    pre = s["b"] + (win * s["w"].t()).sum(1)
    s["state"][idx] = win[:, 1:].to(s["state"].dtype)
    return _silu(pre).to(s["x"].dtype)


def _plain_scan_step(s):
    case, idx = s["case"], s["idx"].long()
    H, G = case["H"], case["G"]
    x, Bm, Cm = (t.float() for t in _split(case, s["xbc"]))
    d = _softplus(s["dt"].float() + s["dt_bias"])
    decay = torch.exp(d * -torch.exp(s["A_log"]))
    Bh, Ch = Bm.repeat_interleave(H // G, 1), Cm.repeat_interleave(H // G, 1)
    st = s["state"][idx] * decay[..., None, None] + Bh[..., None] * (x * d[..., None])[:, :, None]
    s["state"][idx] = st
    y = (st * Ch[..., None]).sum(2) + s["D"][:, None] * x
    return y.to(s["xbc"].dtype)


def _plain_norm(x, res, w):
    h = x if res is None else x + res
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6)
    return h, h * rstd * w


def _plain_quant(y, out, group):
    """8-bit values of y with one scale per row, or per `group` columns of a row."""
    top = 448.0 if out == "e4m3" else 127.0
    cols = y.shape[1]
    size = group or cols
    n = -(-cols // size)
    parts = F.pad(y, (0, n * size - cols)).unflatten(1, (n, size))
    amax = parts.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, amax / top, 1.0)
    q = parts * (1 / scale)
    q = (torch.clamp(q, -top, top).to(torch.float8_e4m3fn) if out == "e4m3"
         else torch.clamp(torch.round(q), -top, top).to(torch.int8))
    return q.flatten(1)[:, :cols], scale[..., 0]


def _values(q, scale, group):
    """What the 8-bit values stand for."""
    cols = q.shape[1]
    wide = scale.repeat_interleave(group or cols, 1)[:, :cols]
    return (q.float() * wide).to(torch.bfloat16)


# --------------------------------------------------------------------------- run
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _dt(case)
    if op == "conv_step":
        return {"y": _plain_conv_step(s), "state": s["state"]}
    if op == "scan_step":
        return {"y": _plain_scan_step(s), "state": s["state"]}
    if op in ("conv", "conv_train"):
        names = ("x", "w", "b", "state")
        ins = [s[k].float() for k in names]
        if op == "conv_train":
            ins = [t.detach().requires_grad_() for t in ins]
        x, w, b, state = ins
        if case["seqs"]:
            y, end = _plain_conv(x[0], w, b, state, s["plan"])
            y = y[None]
        else:
            y, end = _plain_dense_conv(x, w, b, state)
        if op == "conv":
            return {"y": y.to(dt), "state": end.to(dt)}
        dx, dw, db, ds = torch.autograd.grad(y, ins, s["dy"].float())
        return {"y": y.detach().to(dt), "dx": dx.to(dt), "dw": dw, "db": db, "dstate": ds.to(dt)}
    if op in ("scan", "scan_train"):
        flat = [t.flatten(0, 1).float() for t in (*_split(case, s["xbc"]), s["dt"])]
        x, Bm, Cm, d = flat
        ins = [x, d, s["A_log"], Bm, Cm, s["D"], s["dt_bias"], s["h0"]]
        if op == "scan_train":
            ins = [t.detach().requires_grad_() for t in ins]
        y, ht = _plain_scan(*ins, s["plan"])
        lead = (case["B"], case["T"])
        if op == "scan":
            return {"y": y.to(dt).unflatten(0, lead), "ht": ht}
        g = torch.autograd.grad(y, ins, s["dy"].flatten(0, 1).float())
        low = [t.to(dt).unflatten(0, lead) for t in (y.detach(), g[0], g[1], g[3], g[4])]
        return {"y": low[0], "dx": low[1], "ddt": low[2], "dB": low[3], "dC": low[4], "dA_log": g[2],
                "dD": g[5], "ddt_bias": g[6], "dh0": g[7]}
    x, w = s["x"].float(), s["w"]
    res = None if s["res"] is None else s["res"].float()
    if op == "norm":
        h, y = _plain_norm(x, res, w)
        q, scale = _plain_quant(y, case["out"], case["group"])
        return {"h": h.to(dt), "y": _values(q, scale, case["group"]), "scale": scale}
    h, y = _plain_norm(x, res, w)
    # the gradients at the stored (rounded) sum, by the formula
    hs, dy = h.to(dt).float(), s["dy"].float()
    rstd = 1 / torch.sqrt((hs * hs).mean(-1, keepdim=True) + 1e-6)
    xhat, g = hs * rstd, dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True)) + s["dres"].float()
    return {"h": h.to(dt), "y": y.to(dt), "dx": dx.to(dt), "dw": (dy * xhat).sum(0)}


def _run_own(s):
    import gated_delta_rule_cumsum_gb300 as kda

    case = s["case"]
    op = case["op"]
    if op == "conv_step":
        y = kda.short_conv_step(s["x"], s["state"], s["w"], s["b"], state_indices=s["idx"],
                                activation="silu")
        return {"y": y, "state": s["state"]}
    if op == "conv":
        y, end = kda.short_conv(s["x"], s["w"], s["b"], initial_state=s["state"],
                                output_final_state=True, cu_seqlens=s["cu"], activation="silu")
        return {"y": y, "state": end}
    if op == "conv_train":
        kw = dict(initial_state=s["state"], cu_seqlens=s["cu"], activation="silu")
        y, _ = kda.short_conv(s["x"], s["w"], s["b"], **kw)
        g = kda.short_conv_backward(s["x"], s["w"], s["dy"], s["b"], **kw)
        return {"y": y, "dx": g["dx"], "dw": g["dweight"], "db": g["dbias"], "dstate": g["dinitial_state"]}
    if op == "scan_step":
        x, Bm, Cm = _split(case, s["xbc"])
        y = kda.ssm_step(x, s["dt"], s["A_log"], Bm, Cm, s["state"], D=s["D"], dt_bias=s["dt_bias"],
                         dt_softplus=True, state_indices=s["idx"])
        return {"y": y, "state": s["state"]}
    if op in ("scan", "scan_train"):
        x, Bm, Cm = _split(case, s["xbc"])
        kw = dict(D=s["D"], dt_bias=s["dt_bias"], dt_softplus=True, initial_state=s["h0"],
                  cu_seqlens=s["cu"])
        if op == "scan":
            y, ht = kda.ssm_scan(x, s["dt"], s["A_log"], Bm, Cm, output_final_state=True, **kw)
            return {"y": y, "ht": ht}
        y, _, saved = kda.ssm_scan_forward_save(x, s["dt"], s["A_log"], Bm, Cm, **kw)
        g = kda.ssm_scan_backward(x, s["dt"], s["A_log"], Bm, Cm, s["dy"], saved=saved, **kw)
        return {"y": y, "dx": g["dx"], "ddt": g["ddt"], "dB": g["dB"], "dC": g["dC"],
                "dA_log": g["dA_log"], "dD": g["dD"], "ddt_bias": g["ddt_bias"], "dh0": g["dh0"]}
    if op == "norm":
        q, scale, h = kda.add_rms_norm_quant(s["x"], s["w"], residual=s["res"], eps=1e-6,
                                             out_dtype=case["out"], group=case["group"])
        return {"h": h, "y": _values(q, scale, case["group"]), "scale": scale}
    y, h = kda.add_rms_norm(s["x"], s["w"], residual=s["res"], eps=1e-6)
    g = kda.add_rms_norm_backward(s["dy"], h, s["w"], eps=1e-6, dresidual=s["dres"])
    return {"h": h, "y": y, "dx": g["dx"], "dw": g["dweight"]}


# -------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "conv_step":
        n = case["N"] * case["C"]
        return {"bytes": n * e * 2 * case["W"] + case["C"] * 4 * (case["W"] + 1), "flops": n * (2 * case["W"] + 4)}
    if op in ("conv", "conv_train"):
        n, lens, W = case["B"] * case["T"] * case["C"], len(_lens(case)), case["W"]
        state = lens * (W - 1) * case["C"] * e
        if op == "conv":
            return {"bytes": 2 * n * e + 2 * state, "flops": n * (2 * W + 4)}
        return {"bytes": 4 * n * e + 2 * state + 8 * case["C"] * (W + 1), "flops": n * (6 * W + 12)}
    if op.startswith("scan"):
        H, G, P, N = case["H"], case["G"], case["P"], case["N"]
        rows = case["N_seq"] if op == "scan_step" else case["B"] * case["T"]
        seqs = case["N_seq"] if op == "scan_step" else len(_lens(case))
        inputs = rows * (H * P + H + 2 * G * N) * e
        state = seqs * H * N * P * 4
        flops = rows * H * 5 * N * P
        if op == "scan_train":
            return {"bytes": 2 * inputs + 2 * rows * H * P * e + 2 * state, "flops": 3 * flops}
        return {"bytes": inputs + rows * H * P * e + 2 * state, "flops": flops}
    n = case["rows"] * case["cols"]
    ins = (2 if case["residual"] else 1) * e
    if op == "norm":
        groups = -(-case["cols"] // (case["group"] or case["cols"]))
        return {"bytes": n * (ins + e + 1) + case["rows"] * groups * 4, "flops": 8 * n}
    return {"bytes": n * (ins + 2 * e + 3 * e), "flops": 16 * n}


# ------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits: the convolution as a sum over taps of each sequence on
    its own, the scan as the sum over all earlier tokens (no chunks, no state), the step
    and the norm as written."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64

    def one_conv(x, w, b, state):
        ext = torch.cat([state, x])
        win = ext.unfold(0, w.shape[1], 1) if len(x) else ext.new_zeros(0, *w.shape)  # [T, C, W]
        pre = (win * w).sum(-1) + b
        return pre * torch.sigmoid(pre), ext[len(x):]

    def one_scan(x, dt, A_log, Bm, Cm, D, dt_bias, h0, h):
        """One sequence, one head: x [T, P], dt [T], Bm, Cm [T, N], h0 [N, P]."""
        d = torch.logaddexp(dt + dt_bias[h], torch.zeros((), dtype=f64, device=dt.device))
        a = torch.cumsum(-torch.exp(A_log[h]) * d, 0)
        gap = (a[:, None] - a).tril()
        M = (Cm @ Bm.t()).tril() * torch.exp(gap) * d
        y = M @ x + torch.exp(a)[:, None] * (Cm @ h0) + D[h] * x
        left = torch.exp(a[-1] - a) * d
        return y, (Bm * left[:, None]).t() @ x + torch.exp(a[-1]) * h0

    if op == "conv_step":
        idx = s["idx"].long()
        st, x = s["state"].to(f64), s["x"].to(f64)
        pre = s["b"].to(f64) + x * s["w"].to(f64)[:, -1]
        pre = pre + (st[idx] * s["w"].to(f64)[:, :-1].t()).sum(1)
        st[idx] = torch.cat([st[idx][:, 1:], x[:, None]], 1)
        return {"y": pre * torch.sigmoid(pre), "state": st}
    if op in ("conv", "conv_train"):
        train = op == "conv_train"
        x = s["x"].to(f64).flatten(0, 1)
        w, b = s["w"].to(f64).requires_grad_(train), s["b"].to(f64).requires_grad_(train)
        x.requires_grad_(train)
        state = s["state"].to(f64).requires_grad_(train)
        ys, ends, at = [], [], 0
        for i, n in enumerate(_lens(case)):
            y, end = one_conv(x[at:at + n], w, b, state[i])
            ys.append(y)
            ends.append(end)
            at += n
        y = torch.cat(ys).unflatten(0, (case["B"], case["T"]))
        if not train:
            return {"y": y, "state": torch.stack(ends)}
        dx, dw, db, ds = torch.autograd.grad(y, (x, w, b, state), s["dy"].to(f64))
        return {"y": y.detach(), "dx": dx.view_as(y), "dw": dw, "db": db, "dstate": ds}
    if op == "scan_step":
        idx, H, G = s["idx"].long(), case["H"], case["G"]
        x, Bm, Cm = (t.to(f64) for t in _split(case, s["xbc"]))
        d = torch.logaddexp(s["dt"].to(f64) + s["dt_bias"].to(f64), torch.zeros((), dtype=f64, device="cuda"))
        keep = torch.exp(-torch.exp(s["A_log"].to(f64)) * d)
        per = lambda t: t[:, torch.arange(H, device="cuda") // (H // G)]  # noqa: E731
        st = s["state"].to(f64)
        new = keep[..., None, None] * st[idx] + torch.einsum("rh,rhn,rhp->rhnp", d, per(Bm), x)
        st[idx] = new
        y = torch.einsum("rhnp,rhn->rhp", new, per(Cm)) + s["D"].to(f64)[:, None] * x
        return {"y": y, "state": st}
    if op in ("scan", "scan_train"):
        train, H, G = op == "scan_train", case["H"], case["G"]
        x, Bm, Cm = (t.to(f64).flatten(0, 1) for t in _split(case, s["xbc"]))
        dt = s["dt"].to(f64).flatten(0, 1)
        small = [s[k].to(f64).requires_grad_(train) for k in ("A_log", "D", "dt_bias")]
        A_log, D, dt_bias = small
        h0 = s["h0"].to(f64)
        dy = s["dy"].to(f64).flatten(0, 1) if train else None
        y, ht = torch.empty_like(x), h0.clone()
        grads = {k: torch.zeros_like(v) for k, v in (("dx", x), ("ddt", dt), ("dB", Bm), ("dC", Cm),
                                                     ("dA_log", A_log), ("dD", D),
                                                     ("ddt_bias", dt_bias), ("dh0", h0))}
        at = 0
        for i, n in enumerate(_lens(case)):
            r = slice(at, at + n)
            at += n
            for h in range(H if n else 0):
                g = h // (H // G)
                ins = [t.detach().clone().requires_grad_(train)
                       for t in (x[r, h], dt[r, h], Bm[r, g], Cm[r, g], h0[i, h])]
                yy, end = one_scan(ins[0], ins[1], A_log, ins[2], ins[3], D, dt_bias, ins[4], h)
                y[r, h], ht[i, h] = yy.detach(), end.detach()
                if train:
                    got = torch.autograd.grad(yy, [*ins, *small], dy[r, h])
                    grads["dx"][r, h] += got[0]
                    grads["ddt"][r, h] += got[1]
                    grads["dB"][r, g] += got[2]
                    grads["dC"][r, g] += got[3]
                    grads["dh0"][i, h] += got[4]
                    for k, v in zip(("dA_log", "dD", "ddt_bias"), got[5:]):
                        grads[k] += v
        lead = (case["B"], case["T"])
        if not train:
            return {"y": y.unflatten(0, lead), "ht": ht}
        for k in ("dx", "ddt", "dB", "dC"):
            grads[k] = grads[k].unflatten(0, lead)
        return {"y": y.unflatten(0, lead), **{k: v.detach() for k, v in grads.items()}}
    h = s["x"].to(f64) + (0 if s["res"] is None else s["res"].to(f64))
    w = s["w"].to(f64)
    if op == "norm":
        y = h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6) * w
        top, rows, cols = (448.0 if case["out"] == "e4m3" else 127.0), case["rows"], case["cols"]
        size = case["group"] or cols
        q, scales = torch.empty_like(y), []
        for c in range(0, cols, size):
            part = y[:, c:c + size]
            scale = part.abs().amax(1, keepdim=True) / top
            t = part / scale
            if case["out"] == "e4m3":
                # 3 fraction bits, the least exponent -6; ties to even
                step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
                t = torch.round(t / step) * step
            else:
                t = torch.round(t)
            q[:, c:c + size] = t * scale
            scales.append(scale)
        return {"h": h, "y": q, "scale": torch.cat(scales, 1)}
    y = h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6) * w
    hs = h.to(_dt(case)).to(f64).requires_grad_()
    w = w.requires_grad_()
    out = hs / torch.sqrt(hs.pow(2).mean(-1, keepdim=True) + 1e-6) * w
    dx, dw = torch.autograd.grad(out, (hs, w), s["dy"].to(f64))
    return {"h": h, "y": y, "dx": dx + s["dres"].to(f64), "dw": dw}
