"""Host-side checks of a beam search's selection: refusals of the C ABI and of the
binding (no GPU, no compute calls), and pins of the numpy reference."""

import itertools

import numpy as np
import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib
from oracle import beam as R

A = 0x10000       # aligned, never dereferenced
ODD = 0x10002     # not 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    return i8.ensure_built()


def call(lib, logits=A, fp32=0, stride=100, scores=A, live=None, batch=2, beams=3, vocab=100, count=3,
         eos=2, outs=(A, A, A, A), ws=A, wn=1 << 40):
    return lib.i8mm_beam_select(logits, fp32, stride, scores, live, batch, beams, vocab, count, eos,
                                *outs, ws, wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fp32=2), _lib.I8MM_EINVAL), (dict(batch=-1), _lib.I8MM_EINVAL),
    (dict(beams=-1), _lib.I8MM_EINVAL), (dict(vocab=-1), _lib.I8MM_EINVAL),
    (dict(beams=1025), _lib.I8MM_EINVAL), (dict(vocab=(1 << 24) + 1, stride=1 << 25), _lib.I8MM_EINVAL),
    (dict(batch=1 << 23), _lib.I8MM_EINVAL), (dict(batch=1 << 62), _lib.I8MM_EINVAL),
    (dict(count=0), _lib.I8MM_EINVAL), (dict(count=65), _lib.I8MM_EINVAL),
    (dict(stride=99), _lib.I8MM_EINVAL), (dict(stride=1 << 62), _lib.I8MM_EINVAL),
    (dict(eos=-2), _lib.I8MM_EINVAL), (dict(eos=100), _lib.I8MM_EINVAL),
    (dict(logits=None), _lib.I8MM_EINVAL), (dict(logits=A + 1), _lib.I8MM_EALIGN),
    (dict(logits=ODD, fp32=1), _lib.I8MM_EALIGN), (dict(scores=None), _lib.I8MM_EINVAL),
    (dict(scores=ODD), _lib.I8MM_EALIGN), (dict(live=ODD), _lib.I8MM_EALIGN),
    (dict(outs=(None, A, A, A)), _lib.I8MM_EINVAL), (dict(outs=(A, ODD, A, A)), _lib.I8MM_EALIGN),
    (dict(outs=(A, A, None, A)), _lib.I8MM_EINVAL), (dict(outs=(A, A, A, ODD)), _lib.I8MM_EALIGN),
    (dict(ws=None), _lib.I8MM_EWORKSPACE), (dict(wn=8), _lib.I8MM_EWORKSPACE),
    (dict(ws=A + 16), _lib.I8MM_EALIGN)])
def test_refused(lib, kw, status):
    assert call(lib, **kw) == status
    assert lib.i8mm_last_error().startswith(b"i8mm_beam_select: ")


APART = [A + 4096 * i for i in range(6)]   # scores, live and the outputs


@pytest.mark.parametrize("i,j", [(i, j) for i in range(2, 6) for j in range(i)])
def test_outputs_apart(lib, i, j):
    """No output overlaps another or an input, not by its last element either (18
    candidates): the next beams are not written over the last."""
    size = 4 * 2 * (3 if j < 2 else 9)
    for at in (APART[j], APART[j] + size - 4, APART[j] - 4 * 17):
        p = list(APART)
        p[i] = at
        assert call(lib, scores=p[0], live=p[1], count=9, outs=p[2:]) == _lib.I8MM_EINVAL
        assert b"overlaps" in lib.i8mm_last_error()


def test_nothing_to_do_needs_no_device(lib):
    assert call(lib, batch=0, logits=None, scores=None, outs=(None,) * 4, ws=None, wn=0) == _lib.I8MM_OK
    assert lib.i8mm_beam_select_workspace_bytes(0, 0, 3, 100, 3) == 0
    assert lib.i8mm_beam_select_workspace_bytes(0, 2, 3, 100, 65) == 0
    assert lib.i8mm_beam_select_workspace_bytes(0, 2, 3, 100, 3) > 0


@pytest.mark.parametrize("fp32", [0, 1])
def test_workspace_holds_every_piece(lib, fp32):
    """Pieces cover the words, and are at most 65536 of them."""
    for batch, beams, vocab, count in itertools.product((1, 7, 64, 1000), (1, 5, 1024),
                                                        (1, 17, 50257, 1 << 24), (1, 64)):
        need = lib.i8mm_beam_select_workspace_bytes(fp32, batch, beams, vocab, count)
        if batch > (1 << 23) // beams // (vocab // 65536 + 1):
            assert need == 0
            continue
        pieces, rest = divmod(need, batch * beams * 8 * (1 + count))
        assert rest == 0 and -(-vocab // 65536) <= pieces <= max(1024, -(-vocab // 65536))


def test_binding_refusals():
    x, s = torch.zeros((2, 3, 50)), torch.zeros((2, 3))
    with pytest.raises(TypeError):
        i8.beam_select(x.double(), s)
    with pytest.raises(TypeError):
        i8.beam_select(x, s.half())
    with pytest.raises(TypeError):
        i8.beam_select(x, s, torch.ones((2, 3), dtype=torch.bool))
    with pytest.raises(ValueError):
        i8.beam_select(x[0], s)
    with pytest.raises(ValueError):
        i8.beam_select(x, s[:1])
    with pytest.raises(ValueError):
        i8.beam_select(x[:, :, ::2], s)
    with pytest.raises(ValueError):
        i8.beam_select(x[:, 0], s)
    with pytest.raises(ValueError):                       # rows not evenly apart
        i8.beam_select(torch.zeros((2, 4, 50))[:, :3], s)
    with pytest.raises(ValueError):                       # on the host
        i8.beam_select(x, s)


def test_reference_pins():
    """Two words by hand: log softmax of (0, log 3) is (log 1/4, log 3/4)."""
    x = np.log(np.array([[[1.0, 3.0], [1.0, 1.0]]]))
    score, token, parent, live, gap = R.select(x, np.zeros((1, 2)), None, 1, 3)
    assert np.allclose(score, np.log([[3 / 4, 1 / 2, 1 / 2]]))
    assert token.tolist() == [[1, 0, 1]] and parent.tolist() == [[0, 1, 1]]
    assert live.tolist() == [[0, 1, 0]]
    # a beam that has ended stands for itself; one with a NaN for nothing
    x[0, 1, 0] = np.nan
    score, token, parent, live, _ = R.select(x, np.array([[-1.0, 0.0]]), np.array([[0, 1]]), 1, 2)
    assert score.tolist() == [[-1.0, -np.inf]] and token.tolist() == [[1, -1]]
    assert parent.tolist() == [[0, -1]] and live.tolist() == [[0, 0]]


def test_reference_against_every_candidate():
    rng = np.random.default_rng(3)
    x = rng.normal(0, 2, (3, 4, 37)).astype(np.float16)
    s = -rng.random((3, 4)).astype(np.float32) * 5
    score, token, parent, _, _ = R.select(x, s, None, -1, 20)
    z = x.astype(np.float64)
    z = z - np.log(np.exp(z).sum(axis=-1, keepdims=True)) + s[:, :, None]
    for b in range(3):
        order = np.argsort(-z[b].reshape(-1), kind="stable")[:20]
        assert np.allclose(score[b], z[b].reshape(-1)[order])
        assert (parent[b] - 4 * b == order // 37).all() and (token[b] == order % 37).all()
