"""A call's workspace is held until the call returns (no GPU: the tensors stand in host
memory, and nothing is launched)."""

import gc
import types
import weakref

import pytest
import torch

from int8_quantized_matmul_absmax_amd import _lib, ops


class Given:
    """Workspaces that only their call keeps, and whether they were alive in it."""

    def __init__(self):
        self.refs, self.seen = [], 0

    def __call__(self, device, nbytes):
        ws = torch.empty((nbytes,), dtype=torch.uint8)
        self.refs.append(weakref.ref(ws))
        return ws

    def in_call(self):
        gc.collect()
        assert self.refs[-1]() is not None, "the workspace is gone before the kernels are on the stream"
        self.seen += 1


@pytest.fixture
def given(monkeypatch):
    g = Given()
    cpu = torch.device("cpu")
    monkeypatch.setattr(ops, "_on_gpu", lambda **tensors: cpu)
    monkeypatch.setattr(ops, "_run", lambda device, call, *args: g.in_call())
    monkeypatch.setattr(ops, "_raw_stream", lambda device: None)

    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *args: 4096
            return lambda *args: g.in_call() or 0
    monkeypatch.setattr(_lib, "load_library", Library)
    return g


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_beam_select(given):
    ops.beam_select(torch.zeros((1, 2, 50)), torch.zeros((1, 2)), workspace=given)
    assert given.seen == 1


def test_page_tables(given):
    ops.kv_pages_step(ints(3, 5), ints(3), ints(4), 20, 64, workspace=given)
    ops.kv_pages_compact(ints(3, 5), ints(3), 20, 64, workspace=given)
    assert given.seen == 2


def test_attention(given):
    cache = types.SimpleNamespace(device=torch.device("cpu"), kv_heads=2, head_dim=64, ref=None)
    batch = types.SimpleNamespace(device=torch.device("cpu"), total_tokens=3, ref=None)
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    ops.int8_kv_cache_attention_pages(q, ints(3, 2, 5), cache, batch, workspace=given)
    ops.int8_kv_cache_attention(q, cache, batch, workspace=given)
    assert given.seen == 2


def test_given_tensors(given):
    """A tensor is checked and used as it is; its size is the call's to judge."""
    ws = torch.empty(10, dtype=torch.uint8)
    assert ops._scratch(ws, ws.device, None) == (ws, ws.data_ptr(), 10)
    with pytest.raises(TypeError):
        ops._scratch(ws.int(), ws.device, None)
    with pytest.raises(ValueError):
        ops._scratch(ws, torch.device("cuda", 0), None)
    assert ops._scratch(None, ws.device, lambda a: 0, 5) == (None, None, 0)
