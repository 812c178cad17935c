"""The autograd functions of the recurrent block's operators, with the library's calls replaced
by their first-order formulas in torch: what is kept, passed on and refused around the calls.
No GPU is needed."""
import pytest
import torch


@pytest.fixture
def kda(monkeypatch):
    """The package, its operators' calls replaced: y = a x, gradients detached as the library's are."""
    import gated_delta_rule_cumsum_gb300 as kda
    b, log = kda.block, []

    def conv(x, w, bias=None, *, initial_state=None, output_final_state=False, **kw):
        log.append(("conv", kw))
        return x * w.sum(), x[:, -1:].clone()

    def conv_bwd(x, w, dy, bias=None, *, initial_state=None, dfinal_state=None, **kw):
        log.append(("conv_bwd", kw))
        x, w, dy = x.detach(), w.detach(), dy.detach()
        return {"dx": dy * w.sum(), "dweight": (dy * x).sum() * torch.ones_like(w),
                "dbias": None if bias is None else torch.zeros_like(bias), "dinitial_state": None}

    def scan(x, dt, A_log, Bm, Cm, **kw):
        log.append(("scan", kw))
        return x * A_log.sum(), x.new_zeros(1)

    def scan_save(*args, **kw):
        y, ht = scan(*args, **kw)
        return y, ht, torch.arange(64, dtype=torch.uint8)

    def scan_bwd(x, dt, A_log, Bm, Cm, dy, *, dht=None, saved=None, **kw):
        log.append(("scan_bwd", dict(kw, saved=saved)))
        x, A, dy = x.detach(), A_log.detach(), dy.detach()
        g = {k: None for k in ("ddt", "dB", "dC", "dD", "ddt_bias", "dh0")}
        return dict(g, dx=dy * A.sum(), dA_log=(dy * x).sum() * torch.ones_like(A))

    def norm(x, w, *, residual=None, eps=1e-6):
        h = x if residual is None else x + residual
        return h * w, h

    def norm_bwd(dy, h, w, *, eps=1e-6, dresidual=None):
        dy, h, w = dy.detach(), h.detach(), w.detach()
        return {"dx": dy * w + dresidual.detach(), "dweight": (dy * h).sum(0)}

    for name, f in (("short_conv", conv), ("short_conv_backward", conv_bwd), ("ssm_scan", scan),
                    ("ssm_scan_forward_save", scan_save), ("ssm_scan_backward", scan_bwd),
                    ("add_rms_norm", norm), ("add_rms_norm_backward", norm_bwd)):
        monkeypatch.setattr(b, name, f)
    kda.log = log
    yield kda
    del kda.log


def run(kda, which, x, w):
    if which == "conv":
        return kda.short_conv_autograd(x, w)[0]
    if which == "scan":
        z = torch.zeros(1)
        return kda.ssm_scan_autograd(x, z, w, z, z)[0]
    y, h = kda.add_rms_norm_autograd(x, w[0], residual=2 * x if which == "norm_residual" else None)
    return y + h


@pytest.mark.parametrize("which", ["conv", "scan", "norm", "norm_residual"])
@pytest.mark.parametrize("upstream", [False, True])
def test_second_order_gradients_are_refused(kda, which, upstream):
    """A gradient penalty through an operator, beside a loss that has a gradient of its own: the
    penalty's part may not be dropped in silence, whether or not the operator's output gradient
    itself depends on something."""
    x, w = torch.ones(2, 3, requires_grad=True), torch.full((2, 3), 2.0, requires_grad=True)
    y = run(kda, which, x, w)
    loss = (y * y).sum() if upstream else y.sum()
    gx, gw = torch.autograd.grad(loss, (x, w), create_graph=True)
    assert torch.isfinite(gx).all() and torch.isfinite(gw).all()
    for total in ((gx * gx).sum() + (w * w).sum(), gw.sum() + (x * x).sum()):
        with pytest.raises(kda.KdaError) as e:
            torch.autograd.grad(total, (x, w), allow_unused=True, retain_graph=True)
        assert e.value.status == kda.KDA_ERR_UNSUPPORTED and "order" in str(e.value)


@pytest.mark.parametrize("which", ["conv", "scan", "norm", "norm_residual"])
def test_first_order_gradients_stay_as_they_were(kda, which):
    got = []
    for create in (False, True):
        x, w = torch.ones(2, 3, requires_grad=True), torch.full((2, 3), 2.0, requires_grad=True)
        y = run(kda, which, x, w)
        got.append(torch.autograd.grad((y * y).sum(), (x, w), create_graph=create))
        assert all(g.requires_grad == create for g in got[-1])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_chunk_states_are_saved_like_every_tensor(kda):
    """Hooks on saved tensors (checkpointing, offloading) see them, and they go with the graph's
    other tensors once the backward has run."""
    x, A, z = torch.ones(2, 3, requires_grad=True), torch.ones(3, requires_grad=True), torch.zeros(1)
    seen = []

    def pack(t):
        seen.append(t.dtype)
        return t.clone()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y, _ = kda.ssm_scan_autograd(x, z, A, z, z)
    assert torch.uint8 in seen
    node = y.grad_fn
    y.sum().backward(retain_graph=True)
    y.sum().backward()  # the same states twice
    states = [kw["saved"] for name, kw in kda.log if name == "scan_bwd"]
    assert len(states) == 2 and all(torch.equal(t, torch.arange(64, dtype=torch.uint8)) for t in states)
    assert not [v for v in vars(node).values() if isinstance(v, torch.Tensor)]
    with pytest.raises(RuntimeError):
        node.saved_tensors


def test_no_chunk_states_without_saving(kda):
    x, A, z = torch.ones(2, 3, requires_grad=True), torch.ones(3, requires_grad=True), torch.zeros(1)
    kda.ssm_scan_autograd(x, z, A, z, z, save_for_backward=False)[0].sum().backward()
    assert [kw["saved"] for name, kw in kda.log if name == "scan_bwd"] == [None]


def test_status_words_reach_both_directions(kda):
    """Bad offsets and waits that ran out can be read after the forward and after the backward."""
    st = torch.zeros(1, dtype=torch.int32)
    x, w, z = torch.ones(2, 3, requires_grad=True), torch.ones(3, requires_grad=True), torch.zeros(1)
    kda.short_conv_autograd(x, w, dev_status=st)[0].sum().backward()
    kda.ssm_scan_autograd(x, z, w, z, z, dev_status=st)[0].sum().backward()
    kda.short_conv_autograd(x, w)[0].sum().backward()
    assert [(name, kw.get("dev_status") is st) for name, kw in kda.log] == [
        ("conv", True), ("conv_bwd", True), ("scan", True), ("scan_bwd", True), ("conv", False), ("conv_bwd", False)]
