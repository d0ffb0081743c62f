"""gdn_sync_status on the GPU: what gave up is reported once, from whichever kernel, thread or stream it is asked."""
import threading

import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
from gated_deltanet_linear_core_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def test_reports_once_and_clears():
    gdn.gdn_sync_status()
    for _ in range(3):
        gdn.gdn_selftest_bounded_wait(1_000_000)
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_sync_status()
        assert e.value.status == _lib.GDN_ERR_TIMEOUT
        gdn.gdn_sync_status()


def test_many_threads_at_once_of_whom_one_hears():
    """More threads than the words that are kept; the streams are their own."""
    gdn.gdn_sync_status()
    said, n = [], 24
    streams = [torch.cuda.Stream() for _ in range(n)]
    gate = threading.Barrier(n)

    def ask(s):
        for _ in range(20):
            gate.wait()
            try:
                gdn.gdn_sync_status(stream=s)
            except gdn.GDNError as e:
                said.append(e.status)

    threads = [threading.Thread(target=ask, args=(s,)) for s in streams]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert said == []


def test_beside_a_capture_of_another_thread():
    """Asking, for the first time on many threads, neither fails nor spoils another thread's capture of its own calls."""
    x = torch.ones(1000, device="cuda")
    s, side = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(20)]
    graph = torch.cuda.CUDAGraph()
    errors = []

    def ask(stream):
        try:
            gdn.gdn_sync_status(stream=stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s, capture_error_mode="thread_local"):
        y = x * 3
        threads = [threading.Thread(target=ask, args=(t,)) for t in side]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert errors == [] and bool((y == 3).all())
