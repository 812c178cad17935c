"""The recurrent block's operators at sizes where a thread block works on several units, rows or
groups one after another: rings and barriers are used again, operands are replaced, sums run
over a block's units.  Every output against the vectorised fp64 forms of tests/block_reference.py,
and bit for bit against a second call.

On 152 SMs: the scan's state kernel takes 4 to 9 pairs of units a block, its output kernel 8 to 19
units, its gradient kernels 4 to 20, across chunks, groups and sequences; the norm 2 to 17 rows; the
convolution strips of 32 to 128 rows, its step 5 to 19 rows a thread.

Tolerances as in test_gpu_block.py: of each output's largest magnitude.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests import block_reference as ref
from tests.test_gpu_block import F32, LOW, PARAM, offsets, rnd, scan_inputs

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def close(name, got, want, tol=None):
    tol = tol or (LOW if got.dtype == torch.bfloat16 else F32)
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} and {tuple(want.shape)}"
    top, err = float(want.abs().max()), float((got.double() - want).abs().max())
    assert err <= tol * top, f"{name}: {err:.3e} of {top:.3e}, tolerance {tol:.1e}"


def doubles(a):
    return {k: None if v is None else v.double() for k, v in a.items()}


# ------------------------------------------------------------------------- scan
PACKED = [700, 0, 1, 1290, 128, 3, 0, 513, 900, 65, 500]
SCANS = {
    "long": ((64, 1, 128, 64), 1, 4100, None),             # one group: B and C change with the chunk
    "groups": ((64, 4, 128, 64), 1, 4100, None),           # and within it
    "packed": ((64, 2, 128, 64), 1, None, PACKED),
    "two_tiles": ((20, 2, 64, 128), 1, 4100, None),        # two 64-column tiles a head
    "part_tile": ((40, 2, 16, 72), 2, 2300, None),         # the second one of 8 columns
    "odd_groups": ((45, 5, 80, 48), 1, None, PACKED),      # an odd number of units a group: half pairs
}


@pytest.mark.parametrize("which", list(SCANS))
def test_scan(kda_lib, which):
    kda, gen = kda_lib, torch.Generator().manual_seed(len(which))
    (H, G, N, P), B, T, lens = SCANS[which]
    cu = None
    if lens is not None:
        cu, T = offsets(lens)
    seqs = B if lens is None else len(lens)
    a = scan_inputs(gen, (B, T), H, G, N, P, torch.bfloat16)
    h0, dht = rnd(gen, seqs, H, N, P), rnd(gen, seqs, H, N, P)
    dy = rnd(gen, B, T, H, P, dtype=torch.bfloat16)

    def run():
        y, ht, saved = kda.ssm_scan_forward_save(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu)
        g = kda.ssm_scan_backward(**a, dy=dy, initial_state=h0, dht=dht, cu_seqlens=cu, saved=saved)
        return dict(g, y=y, ht=ht)

    got = run()
    (y, ht), r = ref.grads(lambda **k: ref.scan(**k, lens=lens), dict(a, h0=h0), (dy, dht))
    close("y", got["y"], y)
    close("ht", got["ht"], ht)
    for mine, theirs in (("dx", "x"), ("dB", "Bm"), ("dC", "Cm"), ("ddt", "dt"), ("dD", "D"), ("dh0", "h0")):
        close(mine, got[mine], r[theirs])
    for mine, theirs in (("dA_log", "A_log"), ("ddt_bias", "dt_bias")):
        close(mine, got[mine], r[theirs], PARAM)
    for _ in range(2):
        again = run()
        assert all(torch.equal(got[k], again[k]) for k in got)
    plain = kda.ssm_scan(**a, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    assert torch.equal(plain[0], got["y"]) and torch.equal(plain[1], got["ht"])


# ------------------------------------------------------------------------- norm
NORMS = [(5000, 2048), (30000, 256), (2500, 4096), (3000, 1000), (2500, 2049), (1500, 5001), (800, 12000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORMS)
def test_norm(kda_lib, dtype, rows, cols):
    kda, gen = kda_lib, torch.Generator().manual_seed(cols)
    x, res, w = rnd(gen, rows, cols, dtype=dtype), rnd(gen, rows, cols, dtype=dtype, std=2), rnd(gen, cols)
    dy, dh = rnd(gen, rows, cols, dtype=dtype), rnd(gen, rows, cols, dtype=dtype)
    y, h = kda.add_rms_norm(x, w, residual=res)
    wh, wy = ref.norm(x.double(), w.double(), res.double())
    close("h", h, wh)
    close("y", y, wy)
    g = kda.add_rms_norm_backward(dy, h, w, dresidual=dh)
    _, r = ref.grads(lambda h, w: ref.norm(h, w), dict(h=h, w=w), (dh, dy))
    close("dx", g["dx"], r["h"])
    close("dw", g["dweight"], r["w"])
    again = kda.add_rms_norm_backward(dy, h, w, dresidual=dh)
    assert torch.equal(y, kda.add_rms_norm(x, w, residual=res)[0]) and all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind,group", [("e4m3", 128), ("e4m3", 0), ("int8", 128), ("int8", 0)])
@pytest.mark.parametrize("rows,cols", [(1500, 2048), (1300, 4096), (6000, 130), (1300, 1001)])
def test_norm_quantised(kda_lib, dtype, kind, group, rows, cols):
    kda, gen = kda_lib, torch.Generator().manual_seed(cols + group)
    x, w, res = rnd(gen, rows, cols, dtype=dtype), rnd(gen, cols), rnd(gen, rows, cols, dtype=dtype, std=2)
    q, scale, h = kda.add_rms_norm_quant(x, w, residual=res, out_dtype=kind, group=group)
    wh, wy = ref.norm(x.double(), w.double(), res.double())
    close("h", h, wh)
    wq, ws = ob.quantise(wy.cpu().numpy(), kind, group)
    close("scale", scale, torch.from_numpy(ws).cuda())
    off = np.abs(q.float().cpu().numpy().astype(np.float64) - wq)
    # a value within fp32 rounding of a tie may round the other way: one step, and rarely
    step = np.maximum(np.abs(wq) / 8, 2.0 ** -9) if kind == "e4m3" else np.ones_like(wq)
    assert (off <= step * (1 + 1e-12)).all() and (off > 0).mean() <= 1e-3


# ------------------------------------------------------------ short convolution
LONG = [4 * n + n % 3 for n in PACKED]
CONVS = {
    "longest": (6144, 4, 1, 13100, None, torch.bfloat16),   # strips of 64 rows, 128 in the backward
    "dense": (2048, 3, 2, 5000, None, torch.bfloat16),
    "packed": (2056, 4, 1, None, LONG, torch.float32),
    "odd": (1537, 4, 1, None, LONG, torch.bfloat16),      # rows that are not aligned for vectors
    "odd_f32": (1537, 2, 2, 8001, None, torch.float32),
}


@pytest.mark.parametrize("which", list(CONVS))
def test_conv(kda_lib, which):
    kda, gen = kda_lib, torch.Generator().manual_seed(len(which))
    C, W, B, T, lens, dtype = CONVS[which]
    cu = None
    if lens is not None:
        cu, T = offsets(lens)
    seqs = B if lens is None else len(lens)
    x, w, bias = rnd(gen, B, T, C, dtype=dtype), rnd(gen, C, W), rnd(gen, C)
    state, dend = rnd(gen, seqs, W - 1, C, dtype=dtype), rnd(gen, seqs, W - 1, C, dtype=dtype)
    dy = rnd(gen, B, T, C, dtype=dtype)

    def run():
        y, end = kda.short_conv(x, w, bias, initial_state=state, output_final_state=True, cu_seqlens=cu)
        g = kda.short_conv_backward(x, w, dy, bias, initial_state=state, dfinal_state=dend, cu_seqlens=cu)
        return dict(g, y=y, end=end)

    got = run()
    (y, end), r = ref.grads(lambda **k: ref.conv(**k, lens=lens), dict(x=x, w=w, bias=bias, state=state), (dy, dend))
    for name, want in (("y", y), ("end", end), ("dx", r["x"]), ("dweight", r["w"]), ("dbias", r["bias"]),
                       ("dinitial_state", r["state"])):
        close(name, got[name], want)
    again = run()
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,C,W", [(509, 6144, 4), (2003, 6144, 2), (5001, 601, 4), (1701, 2048, 3)])
def test_conv_step(kda_lib, dtype, N, C, W):
    kda, gen = kda_lib, torch.Generator().manual_seed(N)
    slots = N + 7
    x, w, bias = rnd(gen, N, C, dtype=dtype), rnd(gen, C, W), rnd(gen, C)
    cache = rnd(gen, slots, W - 1, C, dtype=dtype)
    idx = torch.randperm(slots, generator=gen)[:N].to(torch.int32).cuda()
    idx[3::50] = -1
    before = cache.clone()
    y = kda.short_conv_step(x, cache, w, bias, state_indices=idx)
    live = idx >= 0
    at = idx[live].long()
    win = torch.cat([before[at], x[live, None]], 1)
    pre = (win.double() * w.double().t()).sum(1) + bias.double()
    want = torch.zeros(N, C, dtype=torch.float64, device="cuda")
    want[live] = pre * torch.sigmoid(pre)
    close("y", y, want)
    after = before.clone()
    after[at] = win[:, 1:]
    assert torch.equal(cache, after) and (y[~live] == 0).all()
