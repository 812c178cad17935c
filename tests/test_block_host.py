"""Host-side refusals of the recurrent block's operators: nothing is enqueued, no GPU is
needed."""
import ctypes

import pytest
import torch

FAKE = 0x1000  # never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_cumsum_gb300 import build as b

    b.build()
    import gated_delta_rule_cumsum_gb300 as kda

    kda.load()
    return kda


def conv(kda, **kw):
    return kda.KdaConvShape(**{**dict(B=1, T=8, C=16, W=4, num_seqs=1, dtype=1, x_stride=0, flags=1), **kw})


def ssm(kda, **kw):
    return kda.KdaSsmShape(**{**dict(B=1, T=8, H=4, G=2, N=16, P=8, num_seqs=1, dtype=1, x_stride=0,
                                     dt_stride=0, b_stride=0, c_stride=0, flags=1), **kw})


def norm(kda, **kw):
    return kda.KdaNormShape(**{**dict(rows=4, cols=16, dtype=1, out=0, group=0, eps=1e-6), **kw})


def said(kda, status, want):
    assert status == want, kda.kda_last_error_message()
    assert kda.kda_last_error_message()


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(C=0), 1), (dict(W=1), 2), (dict(W=5), 2), (dict(num_seqs=2), 1),
    (dict(dtype=9), 1), (dict(flags=4), 2), (dict(x_stride=15), 1), (dict(B=70000, T=70000, num_seqs=70000), 2)])
def test_conv_refusals(kda, kw, status):
    s = ctypes.byref(conv(kda, **kw))
    lib = kda.load()
    said(kda, lib.kda_short_conv_fwd(FAKE, FAKE, None, None, None, s, FAKE, None, None, None), status)
    said(kda, lib.kda_short_conv_bwd(FAKE, FAKE, None, None, None, s, FAKE, None, FAKE, FAKE, None, None,
                                     FAKE, 1 << 30, None, None), status)


def test_conv_pointer_refusals(kda):
    lib, s = kda.load(), ctypes.byref(conv(kda))
    said(kda, lib.kda_short_conv_fwd(FAKE, None, None, None, None, s, FAKE, None, None, None), 1)
    said(kda, lib.kda_short_conv_fwd(FAKE, FAKE, None, FAKE, None, s, FAKE, FAKE, None, None), 1)  # aliased state
    packed = ctypes.byref(conv(kda, B=2, num_seqs=1))
    said(kda, lib.kda_short_conv_fwd(FAKE, FAKE, None, None, FAKE, packed, FAKE, None, None, None), 1)
    need = kda.kda_short_conv_bwd_workspace_size(conv(kda))
    assert need > 0
    said(kda, lib.kda_short_conv_bwd(FAKE, FAKE, None, None, None, s, FAKE, None, FAKE, FAKE, None, None,
                                     FAKE, need - 1, None, None), 1)
    said(kda, lib.kda_short_conv_bwd(FAKE, FAKE, None, None, None, s, FAKE, None, FAKE, FAKE, None, None,
                                     FAKE + 4, need, None, None), 1)
    said(kda, lib.kda_short_conv_step(FAKE, FAKE, None, FAKE, FAKE, 4, s, FAKE, None, None), 1)  # T != 1
    one = ctypes.byref(conv(kda, B=8, T=1, num_seqs=8))
    said(kda, lib.kda_short_conv_step(FAKE, FAKE, None, FAKE, None, 7, one, FAKE, None, None), 1)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(H=3), 1), (dict(G=0), 1), (dict(N=0), 1), (dict(N=257), 2), (dict(P=257), 2),
    (dict(num_seqs=3), 1), (dict(dtype=2), 1), (dict(flags=2), 2), (dict(x_stride=31), 1), (dict(dt_stride=3), 1),
    (dict(b_stride=31), 1), (dict(c_stride=-1), 1)])
def test_ssm_refusals(kda, kw, status):
    s, lib = ssm(kda, **kw), kda.load()
    r = ctypes.byref(s)
    said(kda, lib.kda_ssm_scan_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, None, r, FAKE, None, FAKE,
                                   1 << 40, None, None), status)
    said(kda, lib.kda_ssm_scan_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, None, r, FAKE, None, FAKE,
                                   FAKE, FAKE, FAKE, FAKE, None, None, None, None, FAKE, 1 << 40, None, None),
         status)
    if kw.keys() <= {"B", "H", "G", "N", "P"}:
        assert kda.kda_ssm_workspace_size(s) == 0 and kda.kda_ssm_bwd_workspace_size(s, False) == 0


def test_ssm_no_save(kda):
    """A forward whose workspace the backward will not read needs less of it; the backward
    refuses the flag."""
    flag = kda.KDA_SSM_FLAG_NO_SAVE
    keep, drop = (ssm(kda, B=1, T=300, N=16, P=64, dtype=kda.KDA_DTYPE_BF16, flags=f) for f in (1, 1 | flag))
    assert 0 < kda.kda_ssm_workspace_size(drop) < kda.kda_ssm_workspace_size(keep)
    said(kda, kda.load().kda_ssm_scan_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, None, ctypes.byref(drop),
                                          FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE,
                                          1 << 40, None, None), 1)


def test_ssm_workspace_refusals(kda):
    s, lib = ssm(kda), kda.load()
    r = ctypes.byref(s)
    need, back = kda.kda_ssm_workspace_size(s), kda.kda_ssm_bwd_workspace_size(s, True)
    assert need > 0 and kda.kda_ssm_bwd_workspace_size(s, False) == back + need
    args = (FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, None, r)
    said(kda, lib.kda_ssm_scan_fwd(*args, FAKE, None, FAKE, need - 1, None, None), 1)
    said(kda, lib.kda_ssm_scan_fwd(*args, FAKE, None, FAKE + 16, need, None, None), 1)
    grads = (FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None)
    said(kda, lib.kda_ssm_scan_bwd(*args, *grads, FAKE, FAKE, back - 1, None, None), 1)
    said(kda, lib.kda_ssm_scan_bwd(*args, *grads, FAKE + 16, FAKE, back, None, None), 1)
    said(kda, lib.kda_ssm_step(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, 4, r, FAKE, None, None), 1)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=16385), 2), (dict(dtype=5), 1), (dict(out=3), 1),
    (dict(group=64), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1)])
def test_norm_refusals(kda, kw, status):
    lib, s = kda.load(), ctypes.byref(norm(kda, **kw))
    said(kda, lib.kda_add_rmsnorm_fwd(FAKE, None, FAKE, s, None, FAKE, FAKE, None), status)
    if "out" not in kw and "group" not in kw:
        said(kda, lib.kda_add_rmsnorm_bwd(FAKE, FAKE, FAKE, None, s, FAKE, FAKE, FAKE, 1 << 30, None), status)


def test_norm_pointer_refusals(kda):
    lib = kda.load()
    s = ctypes.byref(norm(kda, out=1))
    said(kda, lib.kda_add_rmsnorm_fwd(FAKE, None, FAKE, s, None, FAKE, None, None), 1)  # no scale
    need = kda.kda_add_rmsnorm_bwd_workspace_size(norm(kda))
    assert need > 0
    s = ctypes.byref(norm(kda))
    said(kda, lib.kda_add_rmsnorm_bwd(FAKE, FAKE, FAKE, None, s, FAKE, FAKE, FAKE, need - 1, None), 1)
    said(kda, lib.kda_add_rmsnorm_bwd(FAKE, FAKE, FAKE, None, s, FAKE, FAKE, FAKE + 8, need, None), 1)


def test_binding_refuses_host_tensors(kda):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: kda.short_conv(x, w), lambda: kda.add_rms_norm(x, torch.ones(8)),
                 lambda: kda.short_conv_step(x[:, 0], torch.zeros(1, 3, 8), w),
                 lambda: kda.ssm_scan(x[..., None], x, torch.zeros(8), x[..., None], x[..., None])):
        with pytest.raises(kda.KdaError):
            call()


def test_rows_are_read_in_place_where_they_can_be(kda):
    rows = kda.block._rows
    wide = torch.zeros(3, 5, 40)
    assert rows(wide, 2) == (wide, 0) or rows(wide, 2)[1] == 0
    part = wide[..., 8:20]
    assert rows(part, 2)[0] is part and rows(part, 2)[1] == 40
    heads = part.unflatten(-1, (3, 4))
    assert rows(heads, 2)[0] is heads and rows(heads, 2)[1] == 40
    for t in (wide.transpose(0, 1), wide[:, ::2], wide[..., ::2], wide[:1].expand(3, 5, 40)):
        got, step = rows(t, 2)
        assert got.is_contiguous() and step == 0 and torch.equal(got, t)
    some = wide[1:2, ::2]  # one sequence: every second row, evenly spaced
    assert rows(some, 2)[0] is some and rows(some, 2)[1] == 80


def test_rows_that_repeat_are_copied(kda):
    """Rows broadcast along a dimension are not evenly spaced: read in place, row b * T + t of
    one row per sequence would lie past the tensor's end."""
    rows = kda.block._rows
    for shape, full in (((3, 1, 8), (3, 5, 8)), ((1, 5, 8), (3, 5, 8)), ((1, 1, 8), (3, 5, 8)),
                        ((3, 1, 2, 4), (3, 5, 2, 4)), ((2, 3, 1, 8), (2, 3, 4, 8))):
        t = torch.arange(float(torch.Size(shape).numel())).view(shape).expand(full)
        got, step = rows(t, 2)
        assert got.is_contiguous() and step == 0 and torch.equal(got, t)
    t = torch.arange(16.).view(2, 8).as_strided((2, 3, 4), (4, 2, 1))  # overlapping rows
    got, step = rows(t, 2)
    assert got.is_contiguous() and step == 0 and torch.equal(got, t)


def test_rows_in_place_stay_inside_their_tensor(kda):
    """Whatever the view, what is read in place are exactly its elements."""
    rows, base = kda.block._rows, torch.arange(4.0 * 6 * 10)
    checked = 0
    for size in ((1, 1, 4), (1, 6, 4), (4, 1, 4), (2, 3, 4), (3, 2, 5), (2, 2, 1)):
        for strides in ((a, b, c) for a in (0, 1, 4, 10, 20, 30, 60) for b in (0, 1, 4, 5, 10, 20) for c in (0, 1, 2)):
            t = base.as_strided(size, strides)
            got, step = rows(t, 2)
            flat = got.as_strided((size[0] * size[1], size[2]), (step or size[2], 1))
            assert torch.equal(flat, t.reshape(-1, size[2])), (size, strides)
            checked += got is t
    assert checked > 20


def strided(n):
    """n bytes by numel(), 16 behind it."""
    return torch.zeros(16, dtype=torch.uint8).expand(n // 16, 16)


def test_binding_refuses_workspaces_with_less_memory_than_elements(kda):
    """The size of a workspace is counted in elements: they have to lie back to back."""
    x, w, rows, half = torch.zeros(1, 8, 16), torch.zeros(16, 4), torch.zeros(4, 16), torch.zeros(16)
    c, n, s = conv(kda, dtype=0), norm(kda, dtype=0), ssm(kda, dtype=0)
    xs, dt, bc, A = torch.zeros(1, 8, 4, 8), torch.zeros(1, 8, 4), torch.zeros(1, 8, 2, 16), torch.zeros(4)
    ins = (xs, dt, A, bc, bc, None, None, None, None, s)
    outs = (xs, None, xs, dt, bc, bc, A, None, None, None)
    calls = [
        lambda ws: kda.kda_short_conv_bwd(x, w, None, None, None, c, x, None, x, w, None, None, ws, stream=FakeStream),
        lambda ws: kda.kda_add_rmsnorm_bwd(rows, rows, half, None, n, rows, half, ws, stream=FakeStream),
        lambda ws: kda.kda_ssm_scan_fwd(*ins, xs, None, ws, stream=FakeStream),
        lambda ws: kda.kda_ssm_scan_bwd(*ins, *outs, None, ws, stream=FakeStream),
    ]
    for call in calls:
        for ws in (strided(1 << 24), torch.zeros(1 << 24, dtype=torch.uint8)[::2]):
            with pytest.raises(kda.KdaError) as e:
                call(ws)
            assert e.value.status == kda.KDA_ERR_INVALID_ARG and "contiguous" in str(e.value)
    whole = torch.zeros(1 << 24, dtype=torch.uint8)
    for saved in (strided(1 << 24), whole[:kda.kda_ssm_workspace_size(s) - 1]):
        with pytest.raises(kda.KdaError) as e:
            kda.kda_ssm_scan_bwd(*ins, *outs, saved, whole, stream=FakeStream)
        assert e.value.status == kda.KDA_ERR_INVALID_ARG and "saved" in str(e.value)


class FakeStream:
    cuda_stream = 0


@pytest.mark.parametrize("word", [torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64),
                                  torch.zeros(0, dtype=torch.int32), torch.zeros(1)])
def test_binding_refuses_other_status_words(kda, word):
    """The kernels write four bytes there."""
    x, w, y = torch.zeros(1, 8, 16), torch.zeros(16, 4), torch.zeros(1, 8, 16)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_short_conv_fwd(x, w, None, None, None, conv(kda, dtype=0), y, None, word, FakeStream)
    assert e.value.status == kda.KDA_ERR_INVALID_ARG and "dev_status" in str(e.value)


@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 128, 2**31 - 255])
def test_ssm_refuses_row_counts_whose_chunk_count_overflows(kda, T):
    """Kernels round rows up to whole chunks (up to 128) in 32 bits."""
    s, lib = ssm(kda, T=T, H=1, G=1, N=8, P=8), kda.load()
    r = ctypes.byref(s)
    assert kda.kda_ssm_workspace_size(s) == 0 and kda.kda_ssm_bwd_workspace_size(s, False) == 0
    said(kda, lib.kda_ssm_scan_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, None, r, FAKE, None, FAKE, 0, None,
                                   None), 2)
    ok = ssm(kda, T=2**31 - 256, H=1, G=1, N=8, P=8)
    assert kda.kda_ssm_workspace_size(ok) > 0


def test_conv_refuses_outputs_over_its_inputs(kda):
    """Strips read the rows before their own while other blocks write theirs."""
    lib, s = kda.load(), ctypes.byref(conv(kda))
    x, y, dy, dx, w, ws = (FAKE * k for k in range(1, 7))
    said(kda, lib.kda_short_conv_fwd(x, w, None, None, None, s, x, None, None, None), 1)
    assert "alias" in kda.kda_last_error_message()
    for out in (x, dy):
        said(kda, lib.kda_short_conv_bwd(x, w, None, None, None, s, dy, None, out, w, None, None, ws, 1 << 30, None,
                                         None), 1)
        assert "alias" in kda.kda_last_error_message()
