"""Waits of the gated delta rule's kernels that run out: KDA_DEVICE_TIMEOUT is reported, the kernels run to
their ends with their copies landed, and the next call on the same memory is right.
KDA_GDN_FLAG_TEST_WAIT_TIMEOUT makes every wait for copies give up at once, while they are on their way.
No GPU fault is involved: the waits are bounded polls of barriers in shared memory."""
import pytest
import torch

from .test_gpu_mixer import delta_inputs, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,T,H,HV,K,V", [
    (torch.bfloat16, 1, 300, 2, 4, 128, 128),     # tensor cores, an SM for every block of a pass
    (torch.bfloat16, 1, 520, 20, 40, 64, 128),    # two blocks of a pass on an SM, units one after another
    (torch.bfloat16, 1, 2100, 16, 16, 64, 64),    # in two parts
    (torch.float32, 2, 130, 2, 4, 40, 24)])       # CUDA cores
def test_waits_that_run_out_are_reported_and_leave_nothing_behind(kda_lib, dtype, B, T, H, HV, K, V):
    kda, gen = kda_lib, torch.Generator().manual_seed(T + HV)
    ins = delta_inputs(gen, B, T, H, HV, K, V, dtype, True)
    do, h0, dht = rnd(gen, B, T, HV, V, dtype=dtype), rnd(gen, B, HV, K, V), rnd(gen, B, HV, K, V)

    def shape(flags):
        return kda.KdaGdnShape(B, T, H, HV, K, V, B, 1 if dtype == torch.bfloat16 else 0, 0.0, 1.0, 0, 0, 0,
                               kda.KDA_GDN_FLAG_QK_L2NORM | flags)

    saved = torch.empty(kda.kda_gdn_workspace_size(shape(0)), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kda.kda_gdn_bwd_workspace_size(shape(0), True), dtype=torch.uint8, device="cuda")
    out = {n: torch.empty_like(t) for n, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0", "o", "ht"),
                                                  (*ins, h0, ins[2], h0))}

    def forward(flags, status):
        kda.kda_gdn_fwd(*ins, h0, None, shape(flags), out["o"], out["ht"], saved, status)

    def backward(flags, status):
        kda.kda_gdn_bwd(*ins, h0, None, shape(flags), do, dht, *[out[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")],
                        saved, ws, status)

    want = None
    for flags in (0, kda.KDA_GDN_FLAG_TEST_WAIT_TIMEOUT, 0):
        for call in (forward, backward):
            if flags and call is backward:
                forward(0, None)
            status = kda.new_status()
            call(flags, status)
            state, bits = kda.kda_read_device_status(status)
            assert (state, bits) == ((kda.KDA_ERR_TIMEOUT, kda.KDA_DEVICE_TIMEOUT) if flags else (kda.KDA_OK, 0))
        got = {n: t.clone() for n, t in out.items()}
        if flags == 0 and want is not None:
            assert all(torch.equal(got[n], want[n]) for n in got)
        want = want or got
