"""The gated delta rule's bf16 outputs are its fp64 results rounded once, next to what two bf16 parts of every
factor leave (tests/test_gpu_mixer.py: SPLIT).  A value that is off by d before its rounding comes out as
a neighbour, one step u away, with probability d / u: the root mean square of that is (d u)^0.5, with u between 2^-8
and 2^-7 of the value.  One part alone anywhere on the way is d = 2^-9 of a term, three times that."""
import numpy as np
import pytest
import torch

from oracle import mixer as om

from .test_gpu_mixer import SPLIT, delta_inputs, f64, rnd

pytestmark = pytest.mark.gpu
ONCE = (SPLIT * 2.0 ** -7.5) ** 0.5


def off(got, want):
    """The norm of got's distance to want rounded to bf16, relative to want's."""
    rounded = f64(torch.from_numpy(want).to(torch.bfloat16))
    return np.linalg.norm(f64(got) - rounded) / np.linalg.norm(want)


@pytest.mark.parametrize("H,HV,K,V", [(1, 1, 128, 128), (2, 4, 128, 128), (1, 2, 64, 128), (2, 2, 72, 40)])
@pytest.mark.parametrize("decay", [0.02, 0.5])
def test_outputs_are_rounded_once(kda_lib, H, HV, K, V, decay):
    kda, gen = kda_lib, torch.Generator().manual_seed(K + V)
    lens = [300, 0, 129, 1]
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    T = sum(lens)
    ins = list(delta_inputs(gen, 1, T, H, HV, K, V, torch.bfloat16, True))
    ins[3] = ins[3] * (decay / 0.2)
    h0 = rnd(gen, len(lens), HV, K, V, std=0.3)
    kw = dict(initial_state=h0, cu_seqlens=cu, qk_l2norm=True)
    o, _ = kda.gated_delta_rule(*ins, **kw)
    ref = [f64(t) for t in ins]
    want, _ = om.gated_delta(*ref, f64(h0), f64(cu).astype(int), l2=True)
    assert off(o, want) <= ONCE
    do, dht = rnd(gen, 1, T, HV, V, dtype=torch.bfloat16), rnd(gen, len(lens), HV, K, V, std=0.3)
    d = kda.gated_delta_backward(*ins, do, dht=dht, **kw)
    want = om.gated_delta_grads(*ref, f64(do), f64(h0), f64(dht), f64(cu).astype(int), l2=True)
    for name in ("dq", "dk", "dv", "dbeta"):
        assert off(d[name], want[name]) <= ONCE, name
