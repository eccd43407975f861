"""The workspace that the layers of a stream share (no GPU: the allocations stand
in host memory)."""

import types

import torch

from int8_quantized_matmul_absmax_amd import linear as L


def test_a_recorded_call_keeps_its_workspace_to_itself(monkeypatch):
    """What a graph recorded must not be the shared tensor, which a larger call
    replaces and frees while the graph's replays still write to it."""
    monkeypatch.setattr(L, "_WORKSPACES", {})
    capturing = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=7))
    eager = L.shared_workspace("cpu", 1000)
    assert L.shared_workspace("cpu", 500) is eager
    capturing.append(True)
    first, second = L.shared_workspace("cpu", 800), L.shared_workspace("cpu", 900)
    assert first.numel() >= 800 and second.numel() >= 900
    capturing.clear()
    shared = {t.data_ptr() for t in L._WORKSPACES.values()}
    assert not shared & {first.data_ptr(), second.data_ptr()}
    assert L.shared_workspace("cpu", 600) is eager          # recording left it as it was
    grown = L.shared_workspace("cpu", 5000)
    assert grown.numel() >= 5000 and L.shared_workspace("cpu", 1000) is grown
