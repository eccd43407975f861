"""Every call runs on its tensors' device, whichever is current (no GPU: the tensors stand
in host memory, and nothing is launched)."""

import types

import pytest
import torch

from int8_quantized_matmul_absmax_amd import _lib, ops

CPU = torch.device("cpu")


@pytest.fixture
def ran(monkeypatch):
    """The names of the library's calls that went through _run, with their device."""
    names = []

    class Library:
        def __getattr__(self, name):
            if name.endswith(("workspace_bytes", "many_outliers")):
                return lambda *args: 4096

            def call(*args):
                raise AssertionError(name + " would run on the current device")
            call.name = name
            return call
    monkeypatch.setattr(_lib, "load_library", Library)
    monkeypatch.setattr(ops, "_on_gpu", lambda **tensors: CPU)
    monkeypatch.setattr(ops, "_raw_stream", lambda device: None)
    monkeypatch.setattr(ops, "_run", lambda device, call, *args: names.append((device, call.name)))
    return names


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_layer_calls(ran):
    x, w = half(3, 32), half(5, 32)
    wq, sw = ops.int8_quantize_colwise_weight(w)
    xq, sx = ops.int8_quantize_rowwise(x)
    ops.outlier_detect_gather(x)
    ops.outlier_detect_quantize(x)
    ops.int8_mm_dequant(xq, wq, sx, sw)
    ops.linear_int8_mixed(x, wq, sw)
    ops.linear_int8_mixed_fp16_weights(x, w, wq, sw)
    ops.gelu_f16(x)
    assert ran == [(CPU, n) for n in (
        "int8_quantize_colwise_weight", "int8_quantize_rowwise", "outlier_detect_gather",
        "outlier_detect_quantize", "int8_mm_dequant", "linear_int8_mixed",
        "linear_int8_mixed_fp16_weights", "i8mm_gelu_f16")]


def test_cache_calls(ran):
    cache = types.SimpleNamespace(device=CPU, kv_heads=2, head_dim=64, ref=None, k_codes=None,
                                  k_means=half(4, 2, 64))
    batch = types.SimpleNamespace(device=CPU, total_tokens=3, ref=None)
    k, q = half(3, 2, 64), half(3, 4, 64)
    pages = torch.zeros((3, 2, 5), dtype=torch.int32)
    ops.int8_kv_cache_append(k, k, cache, batch)
    ops.int8_kv_cache_attention(q, cache, batch)
    ops.int8_kv_cache_read(cache, batch)
    ops.int8_kv_cache_page_means(cache, batch)
    ops.int8_kv_cache_select_pages(q, cache, batch, 5)
    ops.int8_kv_cache_attention_pages(q, pages, cache, batch)
    ops.int8_kv_cache_copy_pages(cache, pages[0, :, :3].contiguous(), pages.view(-1))
    ops.kv_pages_step(pages[0], pages[0, :, 0].contiguous(), pages.view(-1)[:4], 9, 16)
    ops.kv_pages_compact(pages[0], pages[0, :, 0].contiguous(), 9, 16)
    ops.beam_select(torch.zeros((1, 2, 9)), torch.zeros((1, 2)))
    assert ran == [(CPU, n) for n in (
        "int8_kv_cache_append", "int8_kv_cache_attention", "int8_kv_cache_read",
        "int8_kv_cache_page_means", "int8_kv_cache_select_pages", "int8_kv_cache_attention_pages",
        "int8_kv_cache_copy_pages", "i8mm_kv_pages_step_batch", "i8mm_kv_pages_compact",
        "i8mm_beam_select")]


@pytest.mark.parametrize("current", [0, 1])
def test_the_device_is_made_current(monkeypatch, current):
    """And its own stream taken: the default stream's handle is the same on all."""
    now, seen = [current], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *error):
            now[0] = self.before
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ops, "_raw_stream", lambda device: 70 + device.index)
    ops._run(torch.device("cuda", 1), lambda *args: seen.append((now[0], args)) or 0, 5)
    assert seen == [(1, (5, 71))] and now == [current]
