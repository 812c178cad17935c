"""The recurrent block's operators at the edges of their ranges on the GPU: calls without rows,
rows off every vector boundary, values that are not finite, one column."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.test_gpu_block import f64, offsets, rnd, scan_inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- calls without rows
def no_rows(kda, dtype, w, dend, A, dht):
    """The gradients of calls without a single row, whose first kernel is one that otherwise
    comes later."""
    x = torch.empty(2, 0, 24, dtype=dtype, device="cuda")
    c = kda.short_conv_backward(x, w, x, initial_state=dend, dfinal_state=dend)
    d = kda.short_conv_backward(x, w, x)
    n = kda.add_rms_norm_backward(x, x, w[:, 0].contiguous())
    xs, bc = torch.empty(2, 0, 4, 8, dtype=dtype, device="cuda"), torch.empty(2, 0, 2, 16, dtype=dtype, device="cuda")
    s = kda.ssm_scan_backward(xs, xs[..., 0], A, bc, bc, xs, D=A, initial_state=dht, dht=dht)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = kda.ssm_scan_backward(xs[:1], xs[:1, ..., 0], A, bc[:1], bc[:1], xs[:1], D=A, cu_seqlens=cu)
    zeros = [c["dweight"], d["dweight"], n["dweight"], s["dA_log"], s["dD"], p["dA_log"], p["dD"]]
    return zeros, c["dinitial_state"], s["dh0"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_without_rows(kda_lib, dtype):
    """Alone, and in a graph where each follows a copy."""
    gen = torch.Generator().manual_seed(40)
    w, A = torch.randn(24, 4, generator=gen).cuda(), torch.randn(4, generator=gen).cuda()
    dend = torch.randn(2, 3, 24, generator=gen).to(dtype).cuda()
    dht = torch.randn(2, 4, 16, 8, generator=gen).cuda()

    def check(zeros, dstate, dh0):
        assert all((z == 0).all() for z in zeros)
        assert torch.equal(dstate, dend) and torch.equal(dh0, dht)

    check(*no_rows(kda_lib, dtype, w, dend, A, dht))
    torch.cuda.synchronize()
    graph, src = torch.cuda.CUDAGraph(), torch.empty_like(dht)
    with torch.cuda.graph(graph):
        src.copy_(dht)
        zeros, dstate, dh0 = no_rows(kda_lib, dtype, w, dend, A, src)
    for t in (*zeros, dstate, dh0):
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check(zeros, dstate, dh0)


# ------------------------------------------------------------ rows as they lie in memory
def test_repeated_rows(kda_lib):
    """One row for all tokens of several sequences."""
    gen = torch.Generator().manual_seed(41)
    x, w = rnd(gen, 3, 1, 24).expand(3, 9, 24), rnd(gen, 24, 4)
    assert torch.equal(kda_lib.short_conv(x, w)[0], kda_lib.short_conv(x.contiguous(), w)[0])
    a = scan_inputs(gen, (3, 1), 2, 1, 16, 8, torch.float32)
    wide = {k: v.expand(3, 9, *v.shape[2:]) if k in ("x", "dt", "Bm", "Cm") else v for k, v in a.items()}
    whole = {k: v.contiguous() for k, v in wide.items()}
    assert torch.equal(kda_lib.ssm_scan(**wide)[0], kda_lib.ssm_scan(**whole)[0])


def off_by_one(t):
    """A contiguous copy of t one element past an aligned address."""
    if t is None:
        return None
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("H,G,N,P", [(4, 2, 16, 64), (6, 1, 64, 40), (4, 2, 128, 128), (2, 1, 24, 8)])
def test_scan_off_every_vector_boundary(kda_lib, packed, H, G, N, P):
    """bf16 on the tensor cores: x, B and C cut out of odd-width rows at an odd column, every other
    tensor one element past a boundary.  The arithmetic is the aligned call's, in the same order: the
    same bits."""
    kda, gen = kda_lib, torch.Generator().manual_seed(N + P)
    lens = [300, 0, 1, 129, 70]
    cu, T = offsets(lens) if packed else (None, 300)
    B, seqs = (1, len(lens)) if packed else (2, 2)
    a = {k: v.contiguous() for k, v in scan_inputs(gen, (B, T), H, G, N, P, torch.bfloat16).items()}
    h0, dht = rnd(gen, seqs, H, N, P), rnd(gen, seqs, H, N, P)
    dy = rnd(gen, B, T, H, P, dtype=torch.bfloat16)
    y, ht, saved = kda.ssm_scan_forward_save(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    g = kda.ssm_scan_backward(**a, dy=dy, initial_state=h0, dht=dht, cu_seqlens=cu, saved=saved)

    cols = H * P + 2 * G * N
    width = cols + 3 + cols % 2  # odd
    wide = torch.zeros(B, T, width, dtype=torch.bfloat16, device="cuda")
    wide[..., 1:1 + cols] = torch.cat([a[k].flatten(2) for k in ("x", "Bm", "Cm")], -1)
    x, Bm, Cm = wide[..., 1:1 + cols].split([H * P, G * N, G * N], -1)
    ins = (x, off_by_one(a["dt"]), off_by_one(a["A_log"]), Bm, Cm, off_by_one(a["D"]), off_by_one(a["dt_bias"]),
           off_by_one(h0), cu)
    assert width % 2 == 1 and x.data_ptr() % 4 == 2
    shape = kda.KdaSsmShape(B, T, H, G, N, P, seqs, kda.KDA_DTYPE_BF16, width, 0, width, width, 1)
    ws = torch.empty(kda.kda_ssm_workspace_size(shape), dtype=torch.uint8, device="cuda")
    y2, ht2 = off_by_one(torch.zeros_like(y)), off_by_one(torch.zeros_like(ht))
    kda.kda_ssm_scan_fwd(*ins, shape, y2, ht2, ws)
    assert torch.equal(y, y2) and torch.equal(ht, ht2)
    out = {k: off_by_one(torch.zeros_like(v)) for k, v in g.items()}
    for states in (ws, None):
        back = torch.empty(kda.kda_ssm_bwd_workspace_size(shape, states is not None), dtype=torch.uint8, device="cuda")
        kda.kda_ssm_scan_bwd(*ins, shape, off_by_one(dy), off_by_one(dht), out["dx"], out["ddt"], out["dB"], out["dC"],
                             out["dA_log"], out["dD"], out["ddt_bias"], out["dh0"], states, back)
        for k in g:
            assert torch.equal(g[k], out[k]), k
            out[k].zero_()


# ------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_scan_keeps_non_finite_values_to_what_depends_on_them(kda_lib, dtype, bad):
    """Row 100 lies inside a chunk of either path (64 and 128 rows): the rows of its chunk before it
    see it through zeros alone."""
    kda, gen = kda_lib, torch.Generator().manual_seed(42)
    a = scan_inputs(gen, (2, 300), 2, 2, 64, 64, dtype)
    clean, end = kda.ssm_scan(**a, output_final_state=True)

    def spoilt(key, where):
        b = dict(a, **{key: a[key].clone()})
        b[key][where] = bad
        y, ht = kda.ssm_scan(**b, output_final_state=True)
        assert torch.equal(y[1], clean[1]) and torch.equal(y[0, :, 0], clean[0, :, 0]), key
        assert torch.equal(y[0, :100, 1], clean[0, :100, 1]), key
        assert torch.equal(ht[1], end[1]) and torch.equal(ht[0, 0], end[0, 0]), key
        return y[0, :, 1], ht[0, 1]

    rest = [q for q in range(64) if q != 5]
    y, ht = spoilt("x", (0, 100, 1, 5))  # its column from row 100 on
    assert torch.equal(y[:, rest], clean[0, :, 1][:, rest]) and torch.equal(ht[:, rest], end[0, 1][:, rest])
    assert not torch.isfinite(y[100, 5]) and not torch.isfinite(ht[:, 5]).any()
    y, ht = spoilt("Bm", (0, 100, 1, 7))  # a row of the state from there on
    assert not torch.isfinite(y[100]).any() and not torch.isfinite(ht[7]).any()
    others = [n for n in range(64) if n != 7]
    assert torch.equal(ht[others], end[0, 1][others])
    y, ht = spoilt("Cm", (0, 100, 1, 9))  # that row's output alone
    assert not torch.isfinite(y[100]).any() and torch.equal(y[101:], clean[0, 101:, 1])
    assert torch.equal(ht, end[0, 1])
    if bad != float("-inf"):  # (a step of softplus(-inf) is 0)
        y, ht = spoilt("dt", (0, 100, 1))
        assert not torch.isfinite(y[100]).any()


# ------------------------------------------------------------------------- one column
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [True, False])
def test_norm_gradient_of_one_column(kda_lib, dtype, res):
    """dx = rstd (g - xhat mean(g xhat)) + dh, where all but eps cancels.  xhat mean(g xhat) is some
    twelve rounded operations from g, and rstd and its product four more: 24 x 2^-24 of |g rstd|
    bounds what is left of the terms.  The sum that is then rounded to the output's type lies within
    that and its own 2^-24 of the exact one: the output between those two ends, rounded."""
    gen = torch.Generator().manual_seed(43)
    h, w, dy = rnd(gen, 500, 1, dtype=dtype), rnd(gen, 1), rnd(gen, 500, 1, dtype=dtype)
    dh = rnd(gen, 500, 1, dtype=dtype) if res else None
    g = kda_lib.add_rms_norm_backward(dy, h, w, eps=1e-5, dresidual=dh)
    want, wdw = ob.add_rms_norm_grads(f64(h), f64(w), f64(dy), 1e-5, f64(dh))
    terms = np.abs(f64(dy) * f64(w)) / np.sqrt(f64(h) ** 2 + 1e-5)
    room = 24 * 2.0 ** -24 * terms + 2.0 ** -24 * np.abs(want)
    low, high = (f64(torch.from_numpy(want + s * room).to(dtype)) for s in (-1, 1))
    got = f64(g["dx"])
    assert ((low <= got) & (got <= high)).all(), float(np.abs(got - want).max())
    assert np.abs(f64(g["dweight"]) - wdw).max() <= 2e-5 * np.abs(wdw).max()
