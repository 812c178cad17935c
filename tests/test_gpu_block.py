"""GPU parity of the recurrent block's operators (short convolution, state-space scan,
residual RMS norm) against the fp64 loops of oracle/block.py.

Tolerances, of each output's largest magnitude:
  LOW    bf16 outputs: half an ulp is 2^-9 of an element; 2^-8 leaves as much again for the
         fp32 arithmetic behind it (and for sigmoid's fast exponential)
  F32    fp32 outputs: a sum of n terms of one sign is off by at most n 2^-24, and sums here
         have up to a few hundred terms: 2e-5 = 336 x 2^-24
  PARAM  A_log's and dt_bias's gradients: every token's term is a difference of sums over its
         chunk, so each carries about 64 x 2^-22 of the terms it is made of, and those are
         some 20 times the total they leave: 3e-4
"""
import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu
LOW, F32, PARAM = 2.0 ** -8, 2e-5, 3e-4
DTYPES = [torch.bfloat16, torch.float32]


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def close(name, got, want, tol=None):
    tol = tol or (LOW if got.dtype == torch.bfloat16 else F32)
    got = f64(got)
    assert got.shape == want.shape, f"{name}: {got.shape} and {want.shape}"
    top = np.abs(want).max() if want.size else 0.0
    err = np.abs(got - want).max() if want.size else 0.0
    assert err <= tol * top or err == 0, f"{name}: {err:.3e} of {top:.3e}, tolerance {tol:.1e}"


def rnd(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(dtype).cuda()


def offsets(lens, tail=0):
    cu = torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32)
    return cu.cuda(), int(cu[-1]) + tail


BATCHES = {
    "one": (1, 1, None), "two": (2, 2, None), "rows": (3, 37, None), "long": (1, 300, None),
    "packed": (1, None, [1, 0, 2, 3, 0, 70, 129, 5, 0]), "only_empty": (1, None, [0, 0]),
}


def batch(name):
    B, T, lens = BATCHES[name]
    if lens is None:
        return B, T, None, None, B
    cu, T = offsets(lens, tail=6)
    return B, T, cu, f64(cu).astype(int), len(lens)


# ------------------------------------------------------------ short convolution
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", list(BATCHES))
@pytest.mark.parametrize("C,W,silu,extras", [(64, 4, True, True), (13, 3, True, True), (1, 2, False, True),
                                             (520, 4, False, False), (1030, 2, True, False)])
def test_conv(kda_lib, dtype, which, C, W, silu, extras):
    kda, gen = kda_lib, torch.Generator().manual_seed(C + W)
    B, T, cu, cun, N = batch(which)
    x, w = rnd(gen, B, T, C, dtype=dtype), rnd(gen, C, W)
    bias = rnd(gen, C) if extras else None
    state = rnd(gen, N, W - 1, C, dtype=dtype) if extras else None
    act = "silu" if silu else None
    y, end = kda.short_conv(x, w, bias, initial_state=state, output_final_state=True, cu_seqlens=cu,
                            activation=act)
    want, wend = ob.short_conv(f64(x), f64(w), f64(bias), f64(state), cun, silu)
    used = T if cu is None else int(cun[-1])
    close("y", y[:, :used], want[:, :used])
    close("state", end, wend)
    dy = rnd(gen, B, T, C, dtype=dtype)
    dend = rnd(gen, N, W - 1, C, dtype=dtype) if extras else None
    g = kda.short_conv_backward(x, w, dy, bias, initial_state=state, dfinal_state=dend, cu_seqlens=cu,
                                activation=act)
    r = ob.short_conv_grads(f64(x), f64(w), f64(dy), f64(bias), f64(state), f64(dend), cun, silu)
    close("dx", g["dx"], r["dx"])
    close("dw", g["dweight"], r["dw"])
    if extras:
        close("db", g["dbias"], r["db"])
        close("dstate", g["dinitial_state"], r["ds"])
    else:
        assert g["dbias"] is None and g["dinitial_state"] is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [64, 50])
def test_conv_reads_column_ranges_in_place(kda_lib, dtype, C):
    gen = torch.Generator().manual_seed(1)
    wide, w = rnd(gen, 2, 40, C + 30, dtype=dtype), rnd(gen, C, 4)
    x = wide[..., 8:8 + C]
    y, _ = kda_lib.short_conv(x, w)
    assert torch.equal(y, kda_lib.short_conv(x.contiguous(), w)[0])
    odd = wide[..., 5:5 + C]  # rows off any vector boundary
    close("y", kda_lib.short_conv(odd, w)[0], ob.short_conv(f64(odd), f64(w))[0])
    turned = x.transpose(0, 1).contiguous().transpose(0, 1)  # uneven rows: copied
    assert torch.equal(y, kda_lib.short_conv(turned, w)[0])


def test_conv_leaves_rows_outside_alone(kda_lib):
    gen = torch.Generator().manual_seed(2)
    cu, T = offsets([5, 0, 9], tail=4)
    x, w = rnd(gen, 1, T, 24), rnd(gen, 24, 4)
    x[:, 14:] = float("nan")
    y = torch.full((1, T, 24), 7.0, device="cuda")
    kda_lib.kda_short_conv_fwd(x, w, None, None, cu, kda_lib.KdaConvShape(1, T, 24, 4, 3, 0, 0, 1), y, None)
    assert torch.isfinite(y).all() and (y[:, 14:] == 7.0).all()
    g = kda_lib.short_conv_backward(x, w, torch.full_like(x, float("nan")).where(
        torch.arange(T, device="cuda")[:, None] >= 14, torch.ones_like(x)), cu_seqlens=cu)
    assert all(torch.isfinite(t).all() for t in (g["dx"], g["dweight"])) and (g["dx"][:, 14:] == 0).all()


@pytest.mark.parametrize("bad", [[1, 3, 9], [0, 5, 3], [0, 4, 99], [0, -2, 4], [0, 4, -1]])
def test_bad_offsets_are_reported(kda_lib, bad):
    gen = torch.Generator().manual_seed(3)
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x, w = rnd(gen, 1, 12, 8), rnd(gen, 8, 3)
    for call in ("conv", "conv_bwd", "scan", "scan_bwd"):
        st = kda_lib.block._bytes(4, "cuda")[:4].view(torch.int32).zero_()
        if call == "conv":
            kda_lib.short_conv(x, w, cu_seqlens=cu, output_final_state=True, dev_status=st)
        elif call == "conv_bwd":
            kda_lib.short_conv_backward(x, w, x, cu_seqlens=cu, dev_status=st)
        else:
            xs, bc = rnd(gen, 1, 12, 2, 4), rnd(gen, 1, 12, 1, 5)
            args = (xs, rnd(gen, 1, 12, 2), rnd(gen, 2), bc, bc)
            if call == "scan":
                kda_lib.ssm_scan(*args, cu_seqlens=cu, output_final_state=True, dev_status=st)
            else:
                g = kda_lib.ssm_scan_backward(*args, xs, cu_seqlens=cu, dev_status=st)
                assert (g["dx"] == 0).all() and (g["dB"] == 0).all() and (g["dA_log"] == 0).all()
        code, bits = kda_lib.kda_read_device_status(st)
        assert code == kda_lib.KDA_ERR_BAD_CU_SEQLENS and bits & kda_lib.KDA_DEVICE_BAD_CU_SEQLENS, call


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C,W,indexed", [(64, 4, True), (13, 3, True), (600, 2, False), (1, 4, False)])
def test_conv_step_continues_a_prompt(kda_lib, dtype, C, W, indexed):
    kda, gen = kda_lib, torch.Generator().manual_seed(C)
    N, T = 5, 9
    x, w, bias = rnd(gen, N, T, C, dtype=dtype), rnd(gen, C, W), rnd(gen, C)
    want, wend = ob.short_conv(f64(x), f64(w), f64(bias))
    _, end = kda.short_conv(x[:, :T - 3], w, bias, output_final_state=True)
    cache = torch.full((N + 3, W - 1, C), 9.0, dtype=dtype, device="cuda")
    idx = torch.tensor([6, 0, 3, 7, 1], dtype=torch.int32, device="cuda") if indexed else None
    slots = idx.long() if indexed else torch.arange(N, device="cuda")
    cache[slots] = end
    for t in range(T - 3, T):
        y = kda.short_conv_step(x[:, t], cache, w, bias, state_indices=idx)
        close(f"y[{t}]", y, want[:, t])
    close("state", cache[slots], wend)
    rest = torch.ones(N + 3, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert (cache[rest] == 9.0).all()


def test_steps_skip_unused_rows_and_report_bad_indices(kda_lib):
    kda, gen = kda_lib, torch.Generator().manual_seed(5)
    idx = torch.tensor([1, -1, 9, 0], dtype=torch.int32, device="cuda")
    x, w, cache = rnd(gen, 4, 16), rnd(gen, 16, 4), rnd(gen, 2, 3, 16)
    one = cache.clone()
    st = kda.new_status()
    y = kda.short_conv_step(x, cache, w, state_indices=idx, dev_status=st)
    assert (y[1:3] == 0).all() and kda.kda_read_device_status(st)[1] == kda.KDA_DEVICE_BAD_INDEX
    z = kda.short_conv_step(x[[3, 0]], one, w)
    assert torch.equal(z, y[[3, 0]]) and torch.equal(one, cache)
    xs, dt, bc, A = rnd(gen, 4, 2, 8), rnd(gen, 4, 2), rnd(gen, 4, 1, 6), rnd(gen, 2)
    cache = rnd(gen, 2, 2, 6, 8)
    one = cache.clone()
    st = kda.new_status()
    y = kda.ssm_step(xs, dt, A, bc, bc, cache, state_indices=idx, dev_status=st)
    assert (y[1:3] == 0).all() and kda.kda_read_device_status(st)[1] == kda.KDA_DEVICE_BAD_INDEX
    z = kda.ssm_step(xs[[3, 0]], dt[[3, 0]], A, bc[[3, 0]], bc[[3, 0]], one)
    assert torch.equal(z, y[[3, 0]]) and torch.equal(one, cache)


# ------------------------------------------------------------------------- scan
def scan_inputs(gen, lead, H, G, N, P, dtype, strong=False):
    wide = rnd(gen, *lead, H * P + 2 * G * N, dtype=dtype)
    x, Bm, Cm = wide.split([H * P, G * N, G * N], -1)
    a = dict(x=x.unflatten(-1, (H, P)), dt=rnd(gen, *lead, H, dtype=dtype),
             A_log=rnd(gen, H, std=0.7) + (6.0 if strong else 0.5),
             Bm=Bm.unflatten(-1, (G, N)), Cm=Cm.unflatten(-1, (G, N)), D=rnd(gen, H),
             dt_bias=rnd(gen, H) - 2.0)
    return a


SIZES = [(4, 2, 128, 64), (2, 1, 64, 64), (3, 1, 20, 33), (2, 2, 1, 1), (1, 1, 130, 70), (2, 1, 16, 128),
         (2, 2, 128, 192), (1, 1, 256, 256)]


def scan_case(gen, which, sizes, dtype, strong=False):
    H, G, N, P = sizes
    B, T, cu, cun, seqs = batch(which)
    a = scan_inputs(gen, (B, T), H, G, N, P, dtype, strong)
    return a, rnd(gen, seqs, H, N, P), cu, cun, (T if cu is None else int(cun[-1]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", list(BATCHES))
@pytest.mark.parametrize("sizes", SIZES[:3])
def test_scan(kda_lib, dtype, which, sizes):
    check_scan(kda_lib, dtype, which, sizes)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", SIZES[3:])
def test_scan_sizes(kda_lib, dtype, sizes):
    check_scan(kda_lib, dtype, "packed", sizes)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scan_strong_decay(kda_lib, dtype):
    """Steps whose decay underflows within a token: exponents down to about -4000."""
    check_scan(kda_lib, dtype, "long", (2, 1, 64, 64), strong=True)


def check_scan(kda, dtype, which, sizes, strong=False):
    gen = torch.Generator().manual_seed(sum(sizes))
    a, h0, cu, cun, used = scan_case(gen, which, sizes, dtype, strong)
    n = {k: f64(v) for k, v in a.items()}
    y, ht, saved = kda.ssm_scan_forward_save(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    want, wht = ob.ssm_scan(**n, h0=f64(h0), cu=cun)
    close("y", y[:, :used], want[:, :used])
    close("ht", ht, wht)
    dy, dht = rnd(gen, *a["x"].shape, dtype=dtype), rnd(gen, *h0.shape)
    g = kda.ssm_scan_backward(**a, dy=dy, initial_state=h0, dht=dht, cu_seqlens=cu, saved=saved)
    r = ob.ssm_scan_grads(**n, dy=f64(dy), h0=f64(h0), dht=f64(dht), cu=cun)
    for k in ("dx", "dB", "dC", "dh0", "dD"):
        close(k, g[k], r[k])
    close("ddt", g["ddt"], r["ddt"], LOW if dtype == torch.bfloat16 else PARAM)
    for k in ("dA_log", "ddt_bias"):
        close(k, g[k], r[k], PARAM)
    again = kda.ssm_scan_backward(**a, dy=dy, initial_state=h0, dht=dht, cu_seqlens=cu)
    for k in g:  # the same states formed again, the same fixed orders
        assert torch.equal(g[k], again[k]), k


@pytest.mark.parametrize("T", [3, 20, 150])
def test_scan_parameter_gradients_keep_fp32(kda_lib, T):
    """dA_log and ddt_bias are sums of either sign over rows, state rows and columns, and a few
    tokens' are mostly made of the chunk states: these have to enter with fp32's digits.  In
    the 2-norm over 64 heads a sum's own rounding is near 2^-24 a term and the approximate
    exponentials give 2^-22: 1e-6 leaves a factor of four; states of 17 bits would be past 2e-6."""
    gen = torch.Generator().manual_seed(T)
    a = scan_inputs(gen, (1, T), 64, 4, 128, 64, torch.bfloat16)
    h0, dht = rnd(gen, 1, 64, 128, 64), rnd(gen, 1, 64, 128, 64)
    dy = rnd(gen, *a["x"].shape, dtype=torch.bfloat16)
    g = kda_lib.ssm_scan_backward(**a, dy=dy, initial_state=h0, dht=dht)
    r = ob.ssm_scan_grads(**{k: f64(v) for k, v in a.items()}, dy=f64(dy), h0=f64(h0), dht=f64(dht))
    for k in ("dA_log", "ddt_bias"):
        err = np.linalg.norm(f64(g[k]) - r[k]) / np.linalg.norm(r[k])
        assert err <= 1e-6, f"{k}: {err:.2e}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", ["rows", "packed"])
@pytest.mark.parametrize("sizes", [(4, 2, 80, 48), (2, 1, 16, 32), (2, 1, 128, 200), (3, 1, 64, 64), (3, 1, 20, 33)])
def test_scan_whatever_the_workspaces_held(kda_lib, dtype, which, sizes):
    """Workspaces full of NaN (0xff bytes) and of zeros give the same results, bit for bit."""
    H, G, N, P = sizes
    gen = torch.Generator().manual_seed(13)
    a, h0, cu, _, used = scan_case(gen, which, sizes, dtype)
    B, T = a["x"].shape[:2]
    dy, dht = rnd(gen, *a["x"].shape, dtype=dtype), rnd(gen, *h0.shape)
    shape = kda_lib.KdaSsmShape(B, T, H, G, N, P, len(h0), kda_lib.KDA_DTYPE_BF16 if dtype == torch.bfloat16
                                else kda_lib.KDA_DTYPE_F32, 0, 0, 0, 0, 1)
    got = []
    for fill in (0, 255):
        def filled(n):
            return torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        y, ht, saved = kda_lib.ssm_scan_forward_save(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu,
                                                     workspace=filled(kda_lib.kda_ssm_workspace_size(shape)))
        kw = dict(dy=dy, initial_state=h0, dht=dht, cu_seqlens=cu)
        g = kda_lib.ssm_scan_backward(**a, **kw, saved=saved,
                                      workspace=filled(kda_lib.kda_ssm_bwd_workspace_size(shape, True)))
        f = kda_lib.ssm_scan_backward(**a, **kw, workspace=filled(kda_lib.kda_ssm_bwd_workspace_size(shape, False)))
        got.append([y[:, :used], ht, *g.values(), *f.values()])
    for one, other in zip(*got):
        assert torch.isfinite(one).all() and torch.equal(one, other)


def test_other_workspaces_whatever_they_held(kda_lib):
    gen = torch.Generator().manual_seed(14)
    x, dy, w = rnd(gen, 2, 37, 24), rnd(gen, 2, 37, 24), rnd(gen, 24, 4)
    wn, got = rnd(gen, 24), []
    for fill in (0, 255):
        ws = torch.full((1 << 22,), fill, dtype=torch.uint8, device="cuda")
        c = kda_lib.short_conv_backward(x, w, dy, workspace=ws)
        ws = torch.full((1 << 22,), fill, dtype=torch.uint8, device="cuda")
        n = kda_lib.add_rms_norm_backward(dy, x, wn, workspace=ws)
        got.append([c["dx"], c["dweight"], n["dx"], n["dweight"]])
    for one, other in zip(*got):
        assert torch.isfinite(one).all() and torch.equal(one, other)


def test_scan_without_saving_is_the_same(kda_lib):
    gen = torch.Generator().manual_seed(12)
    a, h0, cu, _, used = scan_case(gen, "packed", (2, 1, 64, 64), torch.bfloat16, False)
    y, ht = kda_lib.ssm_scan(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    ys, hs, _ = kda_lib.ssm_scan_forward_save(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    assert torch.equal(y[:, :used], ys[:, :used]) and torch.equal(ht, hs)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scan_without_options(kda_lib, dtype):
    """No D, bias, softplus or initial state; steps that are zero for whole stretches."""
    gen = torch.Generator().manual_seed(11)
    a = scan_inputs(gen, (2, 150), 2, 1, 64, 64, dtype)
    a["D"] = a["dt_bias"] = None
    a["dt"] = a["dt"].abs() * 0.1
    a["dt"][:, 40:110] = 0
    n = {k: f64(v) for k, v in a.items()}
    y, ht = kda_lib.ssm_scan(**a, dt_softplus=False, output_final_state=True)
    want, wht = ob.ssm_scan(**n, softplus=False)
    close("y", y, want)
    close("ht", ht, wht)
    dy = rnd(gen, *a["x"].shape, dtype=dtype)
    g = kda_lib.ssm_scan_backward(**a, dy=dy, dt_softplus=False)
    r = ob.ssm_scan_grads(**n, dy=f64(dy), softplus=False)
    for k in ("dx", "dB", "dC"):
        close(k, g[k], r[k])
    close("ddt", g["ddt"], r["ddt"], LOW if dtype == torch.bfloat16 else PARAM)
    close("dA_log", g["dA_log"], r["dA_log"], PARAM)
    assert g["dD"] is None and g["ddt_bias"] is None and g["dh0"] is None


def test_scan_gradients_against_differences(kda_lib):
    """The kernels' own forward, moved by a little each way, against their gradients (fp32:
    a step of 2^-8 leaves truncation near 2^-16 and rounding near 2^-22 x 2^8 = 2^-14 of the
    loss's terms; 2e-3 of the largest derivative has an order of magnitude in hand)."""
    gen = torch.Generator().manual_seed(12)
    a = scan_inputs(gen, (1, 100), 2, 1, 24, 20, torch.float32)
    h0 = rnd(gen, 1, 2, 24, 20)
    dy = rnd(gen, 1, 100, 2, 20)

    def loss(**kw):
        return float((kda_lib.ssm_scan(**kw)[0].double() * dy.double()).sum())

    g = kda_lib.ssm_scan_backward(**a, dy=dy, initial_state=h0)
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A_log", "dA_log"), ("Bm", "dB"), ("Cm", "dC"),
                      ("D", "dD"), ("dt_bias", "ddt_bias"), ("initial_state", "dh0")):
        base = dict(a, initial_state=h0)
        v = rnd(gen, *base[name].shape)
        e = 2.0 ** -8
        up = loss(**dict(base, **{name: base[name] + e * v}))
        down = loss(**dict(base, **{name: base[name] - e * v}))
        want = (up - down) / (2 * e)
        got = float((g[key].double() * v.double()).sum())
        size = float(g[key].double().norm()) * float(v.double().norm()) / v.numel() ** 0.5
        assert abs(got - want) <= 2e-3 * max(size, abs(want)), (name, got, want)


def test_scan_leaves_rows_outside_alone(kda_lib):
    gen = torch.Generator().manual_seed(13)
    cu, T = offsets([70, 0, 9], tail=5)
    for dtype in DTYPES:
        a = scan_inputs(gen, (1, T), 2, 1, 64, 64, dtype)
        for k in ("x", "dt", "Bm", "Cm"):
            a[k][:, 79:] = float("nan")
        s = kda_lib.KdaSsmShape(1, T, 2, 1, 64, 64, 3, kda_lib.block._code(a["x"]), 256, 0, 256, 256, 1)
        y = torch.full((1, T, 2, 64), 7.0, dtype=dtype, device="cuda")
        ws = torch.empty(kda_lib.kda_ssm_workspace_size(s), dtype=torch.uint8, device="cuda")
        kda_lib.kda_ssm_scan_fwd(a["x"], a["dt"], a["A_log"], a["Bm"], a["Cm"], a["D"], a["dt_bias"], None,
                                 cu, s, y, None, ws)
        assert torch.isfinite(y).all() and (y[:, 79:] == 7.0).all()
        dy = torch.ones((1, T, 2, 64), dtype=dtype, device="cuda")
        dy[:, 79:] = float("nan")
        g = kda_lib.ssm_scan_backward(**a, dy=dy, cu_seqlens=cu)
        assert all(torch.isfinite(v).all() for v in g.values() if v is not None)
        assert all((g[k][:, 79:] == 0).all() for k in ("dx", "ddt", "dB", "dC"))


def test_scan_keeps_non_finite_values_to_their_head_and_time(kda_lib):
    gen = torch.Generator().manual_seed(14)
    for dtype in DTYPES:
        a = scan_inputs(gen, (2, 200), 2, 2, 64, 64, dtype)
        clean = kda_lib.ssm_scan(**a)[0]
        a["x"][0, 100, 1] = float("nan")
        y = kda_lib.ssm_scan(**a)[0]
        assert torch.equal(y[1], clean[1]) and torch.equal(y[0, :, 0], clean[0, :, 0])
        assert torch.isfinite(y[0, :64, 1]).all() and torch.isnan(y[0, 100:, 1]).all()


def test_scan_state_carries_over_and_may_alias(kda_lib):
    gen = torch.Generator().manual_seed(15)
    a = scan_inputs(gen, (1, 333), 2, 1, 64, 64, torch.float32)
    whole, end = kda_lib.ssm_scan(**a, output_final_state=True)
    cut = lambda s: {k: (v[:, s] if k in ("x", "dt", "Bm", "Cm") else v) for k, v in a.items()}  # noqa: E731
    _, mid = kda_lib.ssm_scan(**cut(slice(0, 77)), output_final_state=True)
    rest, last = kda_lib.ssm_scan(**cut(slice(77, 333)), initial_state=mid, output_final_state=True)
    close("y", rest, f64(whole[:, 77:]))
    close("ht", last, f64(end))
    s = kda_lib.KdaSsmShape(1, 333, 2, 1, 64, 64, 1, 0, 256, 0, 256, 256, 1)
    ws = torch.empty(kda_lib.kda_ssm_workspace_size(s), dtype=torch.uint8, device="cuda")
    y, h = torch.empty_like(whole), mid.clone()
    kda_lib.kda_ssm_scan_fwd(a["x"], a["dt"], a["A_log"], a["Bm"], a["Cm"], a["D"], a["dt_bias"], h, None, s,
                             y, h, ws)
    y2, h2 = kda_lib.ssm_scan(**a, initial_state=mid, output_final_state=True)
    assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,indexed", [((4, 2, 128, 64), True), ((3, 1, 20, 33), True),
                                           ((1, 1, 1, 1), False), ((2, 1, 256, 256), False),
                                           ((2, 2, 17, 250), True)])
def test_scan_step_continues_a_prompt(kda_lib, dtype, sizes, indexed):
    kda, gen = kda_lib, torch.Generator().manual_seed(sum(sizes))
    (H, G, N, P), R, T = sizes, 3, 12
    a = scan_inputs(gen, (R, T), H, G, N, P, dtype)
    want, wht = ob.ssm_scan(**{k: f64(v) for k, v in a.items()})
    at = lambda s: {k: (v[:, s] if k in ("x", "dt", "Bm", "Cm") else v) for k, v in a.items()}  # noqa: E731
    _, mid = kda.ssm_scan(**at(slice(0, T - 2)), output_final_state=True)
    cache = torch.full((R + 2, H, N, P), 9.0, device="cuda")
    idx = torch.tensor([4, 0, 3], dtype=torch.int32, device="cuda") if indexed else None
    slots = idx.long() if indexed else torch.arange(R, device="cuda")
    cache[slots] = mid
    for t in range(T - 2, T):
        close(f"y[{t}]", kda.ssm_step(state=cache, state_indices=idx, **at(t)), want[:, t])
    close("state", cache[slots], wht)
    rest = torch.ones(R + 2, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert (cache[rest] == 9.0).all()


# ------------------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 128), (5, 130), (70, 256), (33, 1000), (9, 4096),
                                       (2, 5001), (3, 16384)])
@pytest.mark.parametrize("res", [True, False])
def test_norm(kda_lib, dtype, rows, cols, res):
    kda, gen = kda_lib, torch.Generator().manual_seed(cols)
    x, w = rnd(gen, rows, cols, dtype=dtype), rnd(gen, cols)
    r = rnd(gen, rows, cols, dtype=dtype, std=2) if res else None
    y, h = kda.add_rms_norm(x, w, residual=r, eps=1e-5)
    wh, wy = ob.add_rms_norm(f64(x), f64(w), f64(r), 1e-5)
    close("y", y, wy)
    close("h", h, wh)
    dy, dh = rnd(gen, rows, cols, dtype=dtype), rnd(gen, rows, cols, dtype=dtype) if res else None
    g = kda.add_rms_norm_backward(dy, h, w, eps=1e-5, dresidual=dh)
    wdx, wdw = ob.add_rms_norm_grads(f64(h), f64(w), f64(dy), 1e-5, f64(dh))
    # one column: dx is what the cancellation of g and xhat mean(g xhat) leaves of g rstd
    close("dx", g["dx"], wdx, None if cols > 1 else 1.0)
    close("dw", g["dweight"], wdw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (2, 128), (5, 130), (70, 256), (6, 4096), (2, 5001)])
def test_norm_quantised(kda_lib, dtype, kind, group, rows, cols):
    kda, gen = kda_lib, torch.Generator().manual_seed(cols)
    x, w = rnd(gen, rows, cols, dtype=dtype), rnd(gen, cols)
    r = rnd(gen, rows, cols, dtype=dtype, std=2)
    r[-1], x[-1] = 0, 0  # an all-zero row: scale 1, zeros
    q, scale, h = kda.add_rms_norm_quant(x, w, residual=r, out_dtype=kind, group=group)
    wh, wy = ob.add_rms_norm(f64(x), f64(w), f64(r))
    wq, ws = ob.quantise(wy, kind, group)
    close("h", h, wh)
    close("scale", scale, ws)
    got = f64(q.float())
    # a value within fp32 rounding of a tie may round the other way: one step, and rarely
    off = np.abs(got - wq)
    step = np.maximum(np.abs(wq) / 8, 2.0 ** -9) if kind == "e4m3" else np.ones_like(wq)
    assert (off <= step * (1 + 1e-12)).all()
    assert (off > 0).mean() <= max(1e-3, 1.5 / wq.size)
    assert (scale[-1] == 1).all() and (q[-1].float() == 0).all()


def test_norm_non_finite_rows(kda_lib):
    gen = torch.Generator().manual_seed(20)
    x, w = rnd(gen, 4, 300), rnd(gen, 300)
    clean = kda_lib.add_rms_norm(x, w)[0]
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y = kda_lib.add_rms_norm(x, w)[0]
    assert torch.equal(y[[0, 3]], clean[[0, 3]]) and torch.isnan(y[1]).all()
    for kind in ("e4m3", "int8"):  # int8 has no code for NaN: it shows in the scale
        _, scale, _ = kda_lib.add_rms_norm_quant(x, w, out_dtype=kind)
        assert torch.isnan(scale[[1, 2]]).all() and torch.isfinite(scale[[0, 3]]).all()
        # of the row with the infinity, only its own group (0 inf; the other columns are 0)
        _, scale, _ = kda_lib.add_rms_norm_quant(x, w, out_dtype=kind, group=128)
        assert torch.isnan(scale[1]).all() and torch.isnan(scale[2, 0]) and (scale[2, 1:] == 1).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_norm_quantised_tiny_values(kda_lib, kind):
    """Largest values whose quotient by the top leaves the normal range: the scale stays the
    smallest normal number, and q * scale within half a step of it."""
    x = torch.ones(2, 64, device="cuda")
    w = torch.full((64,), 2.0 ** -125, device="cuda")
    w[1::2] = -(2.0 ** -126)
    q, scale, _ = kda_lib.add_rms_norm_quant(x, w, eps=0.0, out_dtype=kind)
    assert (scale == 2.0 ** -126).all()
    assert torch.equal(q.float(), (w * 2.0 ** 126).expand(2, 64))


def test_norm_gradient_against_differences(kda_lib):
    gen = torch.Generator().manual_seed(21)
    x, w, dy = rnd(gen, 6, 200), rnd(gen, 200), rnd(gen, 6, 200)
    f = lambda x, w: float((kda_lib.add_rms_norm(x, w)[0].double() * dy.double()).sum())  # noqa: E731
    g = kda_lib.add_rms_norm_backward(dy, x, w)
    e = 2.0 ** -7
    for name, key in (("x", "dx"), ("w", "dweight")):
        v = rnd(gen, *(x if name == "x" else w).shape)
        want = ((f(x + e * v, w) - f(x - e * v, w)) if name == "x" else (f(x, w + e * v) - f(x, w - e * v)))
        got = float((g[key].double() * v.double()).sum())
        size = float(g[key].double().norm())
        assert abs(got - want / (2 * e)) <= 2e-3 * max(size, abs(got)), name


# ------------------------------------------------------- the block, streams, graphs
def test_autograd_matches_the_explicit_gradients(kda_lib):
    kda, gen = kda_lib, torch.Generator().manual_seed(30)
    a = scan_inputs(gen, (1, 90), 2, 1, 64, 64, torch.bfloat16)
    h0 = rnd(gen, 1, 2, 64, 64)
    leaves = {k: v.detach().clone().requires_grad_() for k, v in dict(a, initial_state=h0).items()}
    y, ht = kda.ssm_scan_autograd(**leaves)
    dy, dht = rnd(gen, *y.shape, dtype=y.dtype), rnd(gen, *ht.shape)
    torch.autograd.backward([y, ht], [dy, dht])
    g = kda.ssm_scan_backward(**a, dy=dy, initial_state=h0, dht=dht)
    for k, key in (("x", "dx"), ("dt", "ddt"), ("A_log", "dA_log"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"),
                   ("dt_bias", "ddt_bias"), ("initial_state", "dh0")):
        assert torch.equal(leaves[k].grad, g[key]), k
    x, w, b = rnd(gen, 2, 20, 24), rnd(gen, 24, 4), rnd(gen, 24)
    lx, lw, lb = (t.clone().requires_grad_() for t in (x, w, b))
    y, end = kda.short_conv_autograd(lx, lw, lb)
    (y.sum() + end.sum()).backward()
    g = kda.short_conv_backward(x, w, torch.ones_like(x), b, dfinal_state=torch.ones_like(end))
    assert torch.equal(lx.grad, g["dx"]) and torch.equal(lw.grad, g["dweight"]) and torch.equal(lb.grad, g["dbias"])
    x, r, w = rnd(gen, 5, 64), rnd(gen, 5, 64), rnd(gen, 64)
    lx, lr, lw = (t.clone().requires_grad_() for t in (x, r, w))
    y, h = kda.add_rms_norm_autograd(lx, lw, residual=lr)
    (y.sum() + 2 * h.sum()).backward()
    g = kda.add_rms_norm_backward(torch.ones_like(x), h, w, dresidual=torch.full_like(x, 2.0))
    assert torch.equal(lx.grad, g["dx"]) and torch.equal(lr.grad, g["dx"]) and torch.equal(lw.grad, g["dweight"])


def test_side_stream_and_graph_replay(kda_lib):
    kda, gen = kda_lib, torch.Generator().manual_seed(31)
    cu, T = offsets([70, 0, 130])
    a = scan_inputs(gen, (1, T), 2, 1, 128, 64, torch.bfloat16)
    w = rnd(gen, 128, 4)

    def work():
        x, _ = kda.short_conv(a["x"].flatten(2), w, cu_seqlens=cu)
        x = kda.add_rms_norm(x, torch.ones(128, device="cuda"))[0].unflatten(2, (2, 64))
        return kda.ssm_scan(**dict(a, x=x), cu_seqlens=cu, output_final_state=True)

    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, ht = kda.ssm_scan(**a, cu_seqlens=cu, output_final_state=True, stream=side)
    with torch.cuda.stream(side):
        got = work()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.equal(y, kda.ssm_scan(**a, cu_seqlens=cu)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want))
