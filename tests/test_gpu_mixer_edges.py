"""The norms around a gated block at the edges of their ranges: eps = 0, gates far from zero (references are
the fp64 loops of oracle/mixer.py).  How far values that are not finite reach, there and in the gated delta rule."""
import pytest
import torch

from oracle import mixer as om

from .test_gpu_mixer import close, delta_inputs, f64, rnd

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 3, 70])
@pytest.mark.parametrize("cols,group", [(64, 64), (128, 64), (21, 7), (256, 128), (256, 256), (100, 100), (520, 520)])
def test_norms_without_eps(kda_lib, dtype, rows, cols, group):
    """Threads of a block that have no row left must not reach the weights' gradients: with eps = 0 the
    norm of what they hold, zeros, is not a number."""
    kda, gen = kda_lib, torch.Generator().manual_seed(cols + rows)
    x, z, res, dy, dh = (rnd(gen, rows, cols, dtype=dtype) for _ in range(5))
    for w in (rnd(gen, group), rnd(gen, cols)):
        for first in (False, True):
            kw = dict(group=group, activation="silu", gate_first=first, eps=0.0)
            ref = [f64(t) for t in (x, z, w)]
            close("y", kda.gated_rms_norm(x, z, w, **kw), om.gated_norm(*ref, group, "silu", first, 0.0))
            d = kda.gated_rms_norm_backward(dy, x, z, w, **kw)
            want = om.gated_norm_grads(*ref, f64(dy), group, "silu", first, 0.0)
            for name in want:
                close(name, d[name], want[name])
    wa, wb, rs = (rnd(gen, cols) for _ in range(3))
    for gate in (None, "sigmoid"):
        kw = dict(gate=z if gate else None, gate_activation=gate, residual_scale=rs, eps=0.0)
        ref = dict(x=f64(x), res=f64(res), w_post=f64(wa), w_pre=f64(wb), z=f64(kw["gate"]), rs=f64(rs), act=gate, eps=0.0)
        for name, got, want in zip("yh", kda.sandwich_norm(x, res, wa, wb, **kw), om.sandwich(**ref)):
            close(name, got, want)
        d = kda.sandwich_norm_backward(dy, x, res, wa, wb, dresidual_out=dh, **kw)
        want = om.sandwich_grads(**ref, dy=f64(dy), dh=f64(dh))
        for name in want:
            if d[name] is not None:
                close(name, d[name], want[name])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_far_from_zero(kda_lib, dtype, act):
    """Every element next to its own size, the gate's derivative where the sigmoid is next to 1 among them.
    Rows of ones with eps = 0, weights of one and gradients of one leave act(z) and act'(z).

    In units of 2^-24: the exponential and the quotient 4 each (two steps), the sum 1, so 9 for sigmoid(-|z|), as
    many for sigmoid(z) and one for its difference; the product 1 more; z sigmoid(z) and z times the derivative 1
    more, each next to the terms' sizes |sigmoid| + |z sigmoid'|, and their sum 1: less than 16.  bf16: half a step, 2^-8, and next to
    it the fast exponential's 2 + 1.2 |z| steps, 2^-16 up to |z| = 80."""
    kda, gen = kda_lib, torch.Generator().manual_seed(50)
    z = torch.cat([torch.linspace(-20, 20, 1601), torch.randn(383, generator=gen) * 10, torch.linspace(-80, 80, 64)])
    z = z.to(dtype).cuda().view(4, 512)
    one, w = torch.ones_like(z), torch.ones(512, device="cuda")
    z64 = z.double()
    s, e = torch.sigmoid(z64), torch.exp(-z64.abs())
    d = e / (1 + e) ** 2
    a, da = (z64 * s, s + z64 * d) if act == "silu" else (s, d)
    size = s + (z64 * d).abs() if act == "silu" else d
    tol = 16 * 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -16
    y = kda.gated_rms_norm(one, z, w, activation=act, eps=0.0)
    assert ((y.double() - a).abs() <= tol * a.abs()).all()
    got = kda.gated_rms_norm_backward(one, one, z, w, activation=act, eps=0.0)
    assert ((got["dgate"].double() - da).abs() <= tol * size).all()
    # (dL/dh is the residual stream's gradient alone: the second norm's is zero)
    got = kda.sandwich_norm_backward(torch.zeros_like(z), one, one, w, w, dresidual_out=one, gate=z, gate_activation=act,
                                     eps=0.0)
    assert ((got["dgate"].double() - da).abs() <= tol * size).all()


def same_but(got, clean, *touched):
    """got is clean bit for bit outside the index expressions `touched`."""
    a, b = got.clone(), clean.clone()
    for at in touched:
        a[at] = b[at] = 0
    return torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("first", [True, False])
def test_gated_norm_of_values_that_are_not_finite(kda_lib, dtype, bad, first):
    """One value of x, or of the gate: what depends on it is not finite, everything else has the bits it has
    without."""
    kda, gen = kda_lib, torch.Generator().manual_seed(51)
    rows, cols, group = 40, 256, 64
    x, z, dy = (rnd(gen, rows, cols, dtype=dtype) for _ in range(3))
    r, c = 17, 70
    mine = (r, slice(64, 128))  # its group
    for w in (rnd(gen, group), rnd(gen, cols)):
        kw = dict(group=group, gate_first=first)
        y, d = kda.gated_rms_norm(x, z, w, **kw), kda.gated_rms_norm_backward(dy, x, z, w, **kw)
        for which in ("x", "z"):
            b = {"x": x, "z": z}
            b[which] = b[which].clone()
            b[which][r, c] = bad
            yb, db = kda.gated_rms_norm(b["x"], b["z"], w, **kw), kda.gated_rms_norm_backward(dy, b["x"], b["z"], w, **kw)
            alone = which == "z" and not first  # the gate behind the norm: its own column's
            assert same_but(yb, y, (r, c) if alone else mine)
            assert same_but(db["dx"], d["dx"], mine)
            assert same_but(db["dgate"], d["dgate"], (r, c) if alone else mine)
            of = slice(0, group) if len(w) == group else slice(64, 128)
            at = c % group if len(w) == group else c
            assert same_but(db["dweight"], d["dweight"], at if alone else of)
            if bad != bad:
                assert yb[r, c].isnan() and db["dweight"][at].isnan()
                assert (db["dx"][mine].isnan() if which == "x" or first else db["dgate"][r, c].isnan()).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_sandwich_norm_of_values_that_are_not_finite(kda_lib, dtype, bad):
    kda, gen = kda_lib, torch.Generator().manual_seed(52)
    rows, cols, r, c = 40, 200, 17, 70
    ins = {n: rnd(gen, rows, cols, dtype=dtype) for n in ("x", "residual", "gate", "dy", "dh")}
    wa, wb, rs = (rnd(gen, cols) for _ in range(3))

    def run(x, residual, gate, dy, dh):
        kw = dict(gate=gate, gate_activation="silu", residual_scale=rs)
        y, h = kda.sandwich_norm(x, residual, wa, wb, **kw)
        return dict(y=y, h=h, **kda.sandwich_norm_backward(dy, x, residual, wa, wb, dresidual_out=dh, **kw))

    clean = run(**ins)
    for which in ins:
        b = dict(ins)
        b[which] = b[which].clone()
        b[which][r, c] = bad
        got = run(**b)
        for name in ("y", "h", "dx", "dresidual", "dgate"):
            assert same_but(got[name], clean[name], r), (which, name)
        if which in ("residual", "gate"):
            assert same_but(got["h"], clean["h"], (r, c)), which
        if which in ("dy", "dh"):
            assert torch.equal(got["y"], clean["y"]) and torch.equal(got["h"], clean["h"])
        if bad != bad:
            assert got["dx"][r].isnan().all() and (which in ("dy", "dh") or got["y"][r].isnan().all()), which


@pytest.mark.parametrize("dtype,K,V", [(torch.bfloat16, 128, 128), (torch.bfloat16, 64, 32), (torch.float32, 40, 24)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v", "g", "beta", "h0", "do", "dht"])
def test_delta_rule_of_values_that_are_not_finite(kda_lib, dtype, K, V, bad, which):
    """One value of one sequence of three: the other sequences, the value heads that share nothing with it and,
    forward, the chunks before its own keep their bits; what depends on it is not finite."""
    kda, gen = kda_lib, torch.Generator().manual_seed(53)
    H, HV, lens = 2, 4, [140, 400, 77]
    T, t = sum(lens), 140 + 270  # the second sequence's third chunk
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    q, k, v, g, beta = delta_inputs(gen, 1, T, H, HV, K, V, dtype, True)
    h0, dht = rnd(gen, 3, HV, K, V, std=0.3), rnd(gen, 3, HV, K, V, std=0.3)
    ins = dict(q=q, k=k, v=v, g=g, beta=beta, h0=h0, dht=dht, do=rnd(gen, 1, T, HV, V, dtype=dtype))

    def run(q, k, v, g, beta, h0, dht, do):
        kw = dict(initial_state=h0, cu_seqlens=cu, qk_l2norm=True)
        o, ht, saved = kda.gated_delta_forward_save(q, k, v, g, beta, output_final_state=True, **kw)
        return dict(o=o, ht=ht, **kda.gated_delta_backward(q, k, v, g, beta, do, dht=dht, saved=saved, **kw))

    clean = run(**ins)
    b = dict(ins)
    b[which] = b[which].clone()
    at = {"q": (0, t, 1, 3), "k": (0, t, 1, 3), "v": (0, t, 2, 5), "g": (0, t, 2), "beta": (0, t, 2),
          "h0": (1, 2, 3, 5), "dht": (1, 2, 3, 5), "do": (0, t, 2, 5)}[which]
    b[which][at] = bad
    got = run(**b)
    hv = slice(2, 4) if which in "qk" else 2       # value heads, and the head of q and k that they share
    start = 140 if which == "h0" else 140 + 256    # the first row of its chunk (of 128 rows and of 32)
    rows, seq = slice(140, 540), 1
    behind = slice(start, 540)
    if which in ("do", "dht"):
        assert torch.equal(got["o"], clean["o"]) and torch.equal(got["ht"], clean["ht"])
    assert same_but(got["o"], clean["o"], (0, behind, hv))
    assert same_but(got["ht"], clean["ht"], (seq, hv))
    for name in ("dv", "dg", "dbeta"):
        assert same_but(got[name], clean[name], (0, rows, hv)), name
    for name in ("dq", "dk"):
        assert same_but(got[name], clean[name], (0, rows, 1)), name
    assert same_but(got["dinitial_state"], clean["dinitial_state"], (seq, hv))
    if bad != bad:
        if which in ("q", "k", "g", "beta"):
            assert not got["o"][0, t, 2].isfinite().any()
        if which == "v":  # (its own column)
            assert not got["o"][0, t, 2, 5].isfinite()
        if which not in ("q", "do", "dht"):
            assert not got["ht"][seq, 2].isfinite().all()
        name, head = dict(q=("dq", 1), k=("dk", 1), v=("dbeta", 2), g=("dg", 2), beta=("dbeta", 2), h0=("dk", 1),
                          do=("dv", 2), dht=("dv", 2))[which]
        assert not got[name][0, rows, head].isfinite().all()
