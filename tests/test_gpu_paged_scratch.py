"""Scratch that paged attention keeps between eager calls: a host thread's, as long as the thread."""
import gc
import threading

import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from test_gpu_paged import Case, run

pytestmark = pytest.mark.gpu


def _in_thread(work):
    bad = []

    def guarded():
        try:
            work()
        except BaseException as e:                 # noqa: B902  (handed to the test's thread)
            bad.append(e)

    t = threading.Thread(target=guarded)
    t.start()
    t.join()
    assert not bad, bad


def test_scratch_is_given_back_with_its_thread(lla_gpu):
    c = Case([1, 5], [900, 70], 4, 2, 128, 16)
    dev, want = c.device(), run(c)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()

    def work():
        for s in (None, stream):
            with torch.cuda.stream(s):
                out = lla.paged_parallax(**dev)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            del out
        assert torch.cuda.memory_allocated() > before

    for _ in range(3):
        _in_thread(work)
        gc.collect()
        assert torch.cuda.memory_allocated() == before
    lla.lla_sync_status()


def test_more_threads_and_streams_than_one_thread_keeps(lla_gpu):
    """Twelve threads, each on three streams in turn, and ten streams of one thread: the same bits every time."""
    c = Case([1] * 4, [2500, 90, 10, 700], 4, 2, 128, 16, seed=3)
    dev, want = c.device(), run(c)
    streams = [torch.cuda.Stream() for _ in range(10)]
    torch.cuda.synchronize()

    def work(mine, times):
        outs = []
        for _ in range(times):
            for s in mine:
                with torch.cuda.stream(s):
                    outs.append(lla.paged_parallax(**dev))
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)

    bad = []

    def guarded(i):
        try:
            work([streams[(i + k) % 10] for k in range(3)], 20)
        except BaseException as e:                 # noqa: B902
            bad.append(e)

    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(12)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    work(streams, 5)
    lla.lla_sync_status()
