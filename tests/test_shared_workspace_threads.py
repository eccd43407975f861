"""The shared workspace and host threads (no GPU: the allocations stand in host memory)."""

import gc
import threading
import types
import weakref

import torch

from int8_quantized_matmul_absmax_amd import linear as L


def test_threads_do_not_share_a_workspace(monkeypatch):
    """The launches of two threads' calls on one stream may alternate: a workspace that
    both were given would be written by one between the launches of the other."""
    monkeypatch.setattr(L, "_WORKSPACES", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=7))
    mine = L.shared_workspace("cpu", 1000)
    both = threading.Barrier(3)
    got, ended = {}, {}

    def work(name):
        got[name] = L.shared_workspace("cpu", 500), L.shared_workspace("cpu", 400)
        ended[name] = weakref.ref(got[name][0])
        both.wait(60)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    both.wait(60)
    for t in threads:
        t.join()
    assert got[0][0] is got[0][1] and got[1][0] is got[1][1]
    assert len({mine.data_ptr(), got[0][0].data_ptr(), got[1][0].data_ptr()}) == 3
    assert L.shared_workspace("cpu", 1000) is mine
    # what a thread had is dropped with it
    got.clear()
    gc.collect()
    assert all(ref() is None for ref in ended.values())
