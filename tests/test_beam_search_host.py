"""BeamSearch's arguments (no GPU: the tables stand in host memory, nothing is run)."""

import types

import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8


def make(caches, beams=2):
    table = torch.zeros((3, 4), dtype=torch.int32)
    return i8.BeamSearch(i8.KVPages(8, 16), caches, table, torch.zeros(3, dtype=torch.int32), beams)


def test_caches_of_any_iterable():
    """A generator's caches are all checked and all kept: the copies of shared pages are
    made in each of them."""
    good = [types.SimpleNamespace(page_tokens=16, num_pages=8 + i) for i in range(3)]
    assert make(iter(good)).caches == good and make(tuple(good)).caches == good
    assert make(c for c in good).caches == good
    with pytest.raises(ValueError):
        make(iter(good + [types.SimpleNamespace(page_tokens=16, num_pages=7)]))
    for beams in (0, 65):
        with pytest.raises(ValueError):
            make(good, beams)
