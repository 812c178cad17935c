"""The recurrent block's operators at the edges of their ranges on the GPU: calls without rows."""
import pytest
import torch

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
