"""The norms around a gated block at the edges of their ranges: eps = 0, gates far from zero.  References are
the fp64 loops of oracle/mixer.py."""
import pytest
import torch

from oracle import mixer as om

from .test_gpu_mixer import close, f64, rnd

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
