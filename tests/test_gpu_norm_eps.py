"""The residual RMS norm without eps on the GPU."""
import pytest
import torch

from oracle import block as ob
from tests.test_gpu_block import f64, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 3, 70, 700])
@pytest.mark.parametrize("cols", [7, 64, 256, 1000])
def test_gradients_without_eps(kda_lib, dtype, rows, cols):
    """Threads of a block that have no row left must not reach the weight's gradient: with eps = 0 the norm
    of what they hold, zeros, is not a number.  Tolerances, of the largest magnitude: half a step of bf16 and
    as much again; fp32 sums of up to 700 terms, 700^0.5 roundings of 2^-24 of terms up to ten times what
    they leave."""
    gen = torch.Generator().manual_seed(cols + rows)
    h, dy = rnd(gen, rows, cols, dtype=dtype), rnd(gen, rows, cols, dtype=dtype)
    w = rnd(gen, cols)
    d = kda_lib.add_rms_norm_backward(dy, h, w, eps=0.0)
    dx, dw = ob.add_rms_norm_grads(f64(h), f64(w), f64(dy), eps=0.0)
    for name, want in (("dx", dx), ("dweight", dw)):
        tol = 2.0 ** -7 if d[name].dtype == torch.bfloat16 else 2e-5
        assert abs(f64(d[name]) - want).max() <= tol * abs(want).max(), name
