"""The fp64 reference of the recurrent block's operators: closed cases by hand, and its
gradients against central differences."""
import numpy as np
import pytest

from oracle import block as ob


def _inputs(rng, B=1, T=7, H=4, G=2, N=3, P=2):
    return dict(x=rng.normal(size=(B, T, H, P)), dt=rng.normal(size=(B, T, H)),
                A_log=rng.normal(size=H) * 0.5, Bm=rng.normal(size=(B, T, G, N)),
                Cm=rng.normal(size=(B, T, G, N)), D=rng.normal(size=H), dt_bias=rng.normal(size=H))


def _central(f, arrays, name, rng, eps=1e-6):
    """Directional derivative of f along a random direction of arrays[name], and the direction."""
    v = rng.normal(size=arrays[name].shape)
    up, down = dict(arrays), dict(arrays)
    up[name], down[name] = arrays[name] + eps * v, arrays[name] - eps * v
    return (f(up) - f(down)) / (2 * eps), v


@pytest.mark.parametrize("cu,B", [(None, 2), ([0, 3, 3, 4, 7], 1)])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_match_differences(cu, B, softplus):
    rng = np.random.default_rng(0)
    a = _inputs(rng, B=B)
    if not softplus:
        a["dt"], a["dt_bias"] = np.abs(a["dt"]), np.abs(a["dt_bias"])
    n = len(ob.sequences(B, 7, cu))
    a["h0"] = rng.normal(size=(n, 4, 3, 2))
    dy, dht = rng.normal(size=a["x"].shape), rng.normal(size=a["h0"].shape)

    def loss(q):
        y, ht = ob.ssm_scan(**q, cu=cu, softplus=softplus)
        return (y * dy).sum() + (ht * dht).sum()

    g = ob.ssm_scan_grads(**a, dy=dy, dht=dht, cu=cu, softplus=softplus)
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A_log", "dA_log"), ("Bm", "dB"), ("Cm", "dC"),
                      ("D", "dD"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        want, v = _central(loss, a, name, rng)
        assert abs((g[key] * v).sum() - want) <= 1e-6 * max(1, abs(want)), name


@pytest.mark.parametrize("cu", [None, [0, 1, 1, 3, 7]])
@pytest.mark.parametrize("W,silu", [(2, True), (4, True), (3, False)])
def test_conv_gradients_match_differences(cu, W, silu):
    rng = np.random.default_rng(1)
    n = len(ob.sequences(1, 7, cu))
    a = dict(x=rng.normal(size=(1, 7, 3)), w=rng.normal(size=(3, W)), bias=rng.normal(size=3),
             state=rng.normal(size=(n, W - 1, 3)))
    dy, dend = rng.normal(size=a["x"].shape), rng.normal(size=a["state"].shape)

    def loss(q):
        y, end = ob.short_conv(**q, cu=cu, silu=silu)
        return (y * dy).sum() + (end * dend).sum()

    g = ob.short_conv_grads(a["x"], a["w"], dy, a["bias"], a["state"], dend, cu, silu)
    for name, key in (("x", "dx"), ("w", "dw"), ("bias", "db"), ("state", "ds")):
        want, v = _central(loss, a, name, rng)
        assert abs((g[key] * v).sum() - want) <= 1e-6 * max(1, abs(want)), name


def test_norm_gradients_match_differences():
    rng = np.random.default_rng(2)
    a = dict(x=rng.normal(size=(3, 5)), w=rng.normal(size=5), res=rng.normal(size=(3, 5)))
    dy, dh = rng.normal(size=(3, 5)), rng.normal(size=(3, 5))

    def loss(q):
        h, y = ob.add_rms_norm(**q)
        return (y * dy).sum() + (h * dh).sum()

    dx, dw = ob.add_rms_norm_grads(a["x"] + a["res"], a["w"], dy, dh=dh)
    for name, g in (("x", dx), ("res", dx), ("w", dw)):
        want, v = _central(loss, a, name, rng)
        assert abs((g * v).sum() - want) <= 1e-6 * max(1, abs(want)), name


def test_scan_closed_forms():
    rng = np.random.default_rng(3)
    a = _inputs(rng)
    h0 = rng.normal(size=(1, 4, 3, 2))
    # no step: the state stays and is read out
    y, ht = ob.ssm_scan(a["x"], np.zeros_like(a["dt"]), a["A_log"], a["Bm"], a["Cm"], h0=h0, softplus=False)
    assert np.array_equal(ht, h0)
    assert np.allclose(y[0, 2, 3], h0[0, 3].T @ a["Cm"][0, 2, 1])
    # one token from nothing: y = d (C . B) x + D x
    one = {k: (v[:, :1] if k in ("x", "dt", "Bm", "Cm") else v) for k, v in a.items()}
    y, _ = ob.ssm_scan(**one)
    d = np.log1p(np.exp(one["dt"][0, 0] + a["dt_bias"]))
    dot = (one["Cm"][0, 0] * one["Bm"][0, 0]).sum(-1)[np.arange(4) // 2]
    assert np.allclose(y[0, 0], (d * dot + a["D"])[:, None] * one["x"][0, 0])


def test_conv_state_carries_over():
    rng = np.random.default_rng(4)
    x, w = rng.normal(size=(1, 9, 3)), rng.normal(size=(3, 4))
    whole, _ = ob.short_conv(x, w)
    first, mid = ob.short_conv(x[:, :2], w)
    rest, _ = ob.short_conv(x[:, 2:], w, state=mid)
    assert np.allclose(np.concatenate([first, rest], 1), whole)


def test_e4m3_rounding_table():
    v = np.array([0.0, 2.0 ** -9, 2.0 ** -10, 1.0625, 1.1875, 447.0, 448.0, 500.0, -17.0])
    assert np.array_equal(ob.round_e4m3(v), [0, 2.0 ** -9, 0, 1.0, 1.25, 448, 448, 448, -16.0])
