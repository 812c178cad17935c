"""Calls of the gated delta rule that are made at once: on streams one of which stands still, from two host
threads.  The calls are long enough to be cut in two parts, one of which runs on a stream of the library's own."""
import threading

import pytest
import torch

from .test_gpu_mixer import delta_inputs, rnd
from .test_gpu_mixer_long import both_ways

pytestmark = pytest.mark.gpu
B, T, H, HV, K, V = 2, 2100, 16, 16, 64, 32


def call_of(gen):
    ins = delta_inputs(gen, B, T, H, HV, K, V, torch.bfloat16, True)
    return ins, rnd(gen, B, T, HV, V, dtype=torch.bfloat16), rnd(gen, B, HV, K, V), rnd(gen, B, HV, K, V)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_call_does_not_wait_for_another_streams(kda_lib):
    """A call behind 0.2 s of another kernel's work, then one on a free stream: the second is through first."""
    gen = torch.Generator().manual_seed(6)
    calls, streams = [call_of(gen) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    want = [both_ways(kda_lib, *c, qk_l2norm=True) for c in calls]
    torch.cuda.synchronize()
    for s, c in zip(streams, calls):  # (their allocations are made)
        with torch.cuda.stream(s):
            both_ways(kda_lib, *c, qk_l2norm=True)
    torch.cuda.synchronize()
    got, stood = [], torch.cuda.Event()
    for n, (s, c) in enumerate(zip(streams, calls)):
        with torch.cuda.stream(s):
            if n == 0:
                torch.cuda._sleep(400_000_000)
                stood.record()
            got.append(both_ways(kda_lib, *c, qk_l2norm=True))
    streams[1].synchronize()
    assert not stood.query()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))


def test_more_streams_at_once_than_the_library_has(kda_lib):
    """Eight calls behind as many waits: those that find no stream of the library's free run in one part."""
    gen = torch.Generator().manual_seed(7)
    calls, streams = [call_of(gen) for _ in range(8)], [torch.cuda.Stream() for _ in range(8)]
    want = [both_ways(kda_lib, *c, qk_l2norm=True) for c in calls]
    torch.cuda.synchronize()
    got = []
    for s, c in zip(streams, calls):
        with torch.cuda.stream(s):
            torch.cuda._sleep(40_000_000)
            got.append(both_ways(kda_lib, *c, qk_l2norm=True))
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))


def test_two_host_threads(kda_lib):
    """Each on its own stream with its own inputs, again and again: the bits of the calls made alone; and
    both on one stream."""
    gen = torch.Generator().manual_seed(8)
    calls = [call_of(gen) for _ in range(2)]
    want = [both_ways(kda_lib, *c, qk_l2norm=True) for c in calls]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    for streams in ([torch.cuda.Stream() for _ in range(2)], [one, one]):
        barrier, errors = threading.Barrier(2), []

        def work(n):
            try:
                torch.cuda.set_device(0)
                barrier.wait()
                for _ in range(20):
                    with torch.cuda.stream(streams[n]):
                        got = both_ways(kda_lib, *calls[n], qk_l2norm=True)
                        ok = torch.stack([(x == y).all() for x, y in zip(got, want[n])]).all()
                    streams[n].synchronize()
                    assert ok.item()
            except BaseException as e:  # noqa: BLE001
                errors.append(repr(e))

        threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not errors, errors


def test_no_wait_runs_out_beside_other_calls(kda_lib):
    """Blocks of several kernels on an SM hold each other's threads up: a thread that comes late to a wait
    must still find its phase."""
    gen = torch.Generator().manual_seed(9)
    calls, streams = [call_of(gen) for _ in range(3)], [torch.cuda.Stream() for _ in range(3)]
    status = [kda_lib.new_status() for _ in calls]
    want = [both_ways(kda_lib, *c, qk_l2norm=True) for c in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[] for _ in calls]
        for _ in range(4):
            for n, (s, c) in enumerate(zip(streams, calls)):
                with torch.cuda.stream(s):
                    got[n].append(both_ways(kda_lib, *c, qk_l2norm=True, dev_status=status[n]))
        torch.cuda.synchronize()
        assert all(kda_lib.kda_read_device_status(w) == (kda_lib.KDA_OK, 0) for w in status)
        for n in range(3):
            assert all(same(g, want[n]) for g in got[n])
