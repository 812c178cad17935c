"""The vectorised fp64 forms of tests/block_reference.py against the token loops of oracle/block.py.
Both are fp64: sums of a few hundred terms agree to 1e-11 of the largest."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests import block_reference as ref


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float64)


def same(got, want):
    got = got.numpy()
    assert got.shape == want.shape and np.abs(got - want).max() <= 1e-11 * max(np.abs(want).max(), 1e-30)


@pytest.mark.parametrize("B,T,lens", [(2, 70, None), (1, 150, [1, 0, 130, 3, 9])])
def test_scan(B, T, lens):
    gen, (H, G, P, N) = torch.Generator().manual_seed(1), (4, 2, 5, 3)
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)])
    seqs = B if lens is None else len(lens)
    a = dict(x=rnd(gen, B, T, H, P), dt=rnd(gen, B, T, H), A_log=rnd(gen, H), Bm=rnd(gen, B, T, G, N),
             Cm=rnd(gen, B, T, G, N), D=rnd(gen, H), dt_bias=rnd(gen, H), h0=rnd(gen, seqs, H, N, P))
    dy, dht = rnd(gen, B, T, H, P), rnd(gen, seqs, H, N, P)
    (y, ht), g = ref.grads(lambda **k: ref.scan(**k, lens=lens), a, (dy, dht))
    n = {k: v.numpy() for k, v in a.items()}
    wy, wht = ob.ssm_scan(**n, cu=cu)
    same(y, wy)
    same(ht, wht)
    r = ob.ssm_scan_grads(**n, dy=dy.numpy(), dht=dht.numpy(), cu=cu)
    for mine, theirs in (("x", "dx"), ("dt", "ddt"), ("A_log", "dA_log"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"),
                         ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        same(g[mine], r[theirs])


@pytest.mark.parametrize("B,T,lens", [(2, 9, None), (1, 20, [1, 0, 12, 2])])
@pytest.mark.parametrize("silu", [True, False])
def test_conv(B, T, lens, silu):
    gen, (C, W) = torch.Generator().manual_seed(2), (5, 4)
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)])
    seqs = B if lens is None else len(lens)
    a = dict(x=rnd(gen, B, T, C), w=rnd(gen, C, W), bias=rnd(gen, C), state=rnd(gen, seqs, W - 1, C))
    dy, dend = rnd(gen, B, T, C), rnd(gen, seqs, W - 1, C)
    (y, end), g = ref.grads(lambda **k: ref.conv(**k, lens=lens, silu=silu), a, (dy, dend))
    n = {k: v.numpy() for k, v in a.items()}
    wy, wend = ob.short_conv(n["x"], n["w"], n["bias"], n["state"], cu, silu)
    same(y, wy)
    same(end, wend)
    r = ob.short_conv_grads(n["x"], n["w"], dy.numpy(), n["bias"], n["state"], dend.numpy(), cu, silu)
    for mine, theirs in (("x", "dx"), ("w", "dw"), ("bias", "db"), ("state", "ds")):
        same(g[mine], r[theirs])


def test_norm():
    gen = torch.Generator().manual_seed(3)
    x, res, w, dy, dh = (rnd(gen, 6, 9), rnd(gen, 6, 9), rnd(gen, 9), rnd(gen, 6, 9), rnd(gen, 6, 9))
    (h, y), g = ref.grads(lambda x, w, res: ref.norm(x, w, res, 1e-5), dict(x=x, w=w, res=res), (dh, dy))
    wh, wy = ob.add_rms_norm(x.numpy(), w.numpy(), res.numpy(), 1e-5)
    same(h, wh)
    same(y, wy)
    wdx, wdw = ob.add_rms_norm_grads(wh, w.numpy(), dy.numpy(), 1e-5, dh.numpy())
    same(g["x"], wdx)
    same(g["res"], wdx)
    same(g["w"], wdw)
