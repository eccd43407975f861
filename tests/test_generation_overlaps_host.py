"""Outputs and workspaces of beam selection and page tables that share memory with what
the call reads or writes elsewhere are refused (no GPU: the addresses are never used)."""

import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib
from tests.test_kv_pages_full_host import APART, call

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    return i8.ensure_built()


def beam(lib, outs, fp32=0, logits=A, stride=100, ws=1 << 31, live=3 << 28):
    """2 searches of 3 beams of 100 words, 9 places."""
    return lib.i8mm_beam_select(logits, fp32, stride, 1 << 28, live, 2, 3, 100, 9, 2, *outs, ws, 1 << 20,
                                None)


def refused(lib, status):
    return status == _lib.I8MM_EINVAL and b"overlaps" in lib.i8mm_last_error()


@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("fp32,stride", [(0, 100), (1, 100), (0, 333), (1, 4000)])
def test_beams_written_over_logits(lib, i, fp32, stride):
    outs = [(2 + j) << 28 for j in (2, 3, 4, 5)]
    span = (5 * stride + 100) * (4 if fp32 else 2)
    for at in (A, A + 4, A + (span - 1) // 4 * 4, A - 4 * 17):
        outs[i] = at
        assert refused(lib, beam(lib, outs, fp32, stride=stride)), at
    for at in (A + (span + 3) // 4 * 4, A - 4 * 18):
        outs[i] = at
        assert not refused(lib, beam(lib, outs, fp32, stride=stride)), at


@pytest.mark.parametrize("at", range(7))
def test_workspaces_of_beams(lib, at):
    """Over logits, scores, live or an output, with its first byte or its last."""
    need = lib.i8mm_beam_select_workspace_bytes(0, 2, 3, 100, 9)
    places = [A, 1 << 28, 3 << 28, 4 << 28, 5 << 28, 6 << 28, 7 << 28]
    assert beam(lib, places[3:]) == _lib.I8MM_ENODEVICE
    assert refused(lib, beam(lib, places[3:], ws=places[at]))
    assert refused(lib, beam(lib, places[3:], ws=places[at] - (need - 1) // 256 * 256))
    assert not refused(lib, beam(lib, places[3:], ws=places[at] - (need + 255) // 256 * 256))


@pytest.mark.parametrize("name", APART)
def test_workspaces_of_page_tables(lib, name):
    apart = {n: (1 + i) << 28 for i, n in enumerate(APART)}
    for ws in (apart[name], apart[name] - 256 * 600):
        assert refused(lib, call(lib, pages=20000, ws=ws, **apart))
    assert not refused(lib, call(lib, pages=20000, ws=apart[name] - (1 << 20), **apart))
    # what one block does needs no workspace, whatever is given
    assert not refused(lib, call(lib, ws=apart[name], **apart))

    def compact(ws):
        return lib.i8mm_kv_pages_compact(apart["table"], apart["lens"], 3, 5, 20000, 64, apart["out"],
                                         apart["copies"], apart["counts"], ws, 1 << 40, None)
    if name in ("table", "lens", "out", "copies", "counts"):
        assert refused(lib, compact(apart[name])) and refused(lib, compact(apart[name] - 256 * 600))
    assert not refused(lib, compact(apart[name] - (1 << 20)))
