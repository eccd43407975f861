"""A beam search's selection on the GPU against the numpy reference."""

import numpy as np
import pytest
import torch

from oracle import beam as R
from tests.gpu_helpers import dev, host, note

pytestmark = pytest.mark.gpu

# A value is the score and the logit, both exact, less the logarithm of a sum that
# is within 2^-18 of itself; then one rounding to fp32.
SUM = 2.0 ** -18


def check(i8, x, scores, live=None, eos=2, count=None, workspace=None, equal_beams=False):
    count = x.shape[1] if count is None else count
    *want, gap = R.select(x if isinstance(x, np.ndarray) else host(x), scores, live, eos, count)
    # each value may be off by SUM: no choice that this could turn (equal beams' sums
    # are equal, whatever they are off by)
    assert gap.min() > 2 * SUM or equal_beams, gap.min()
    out = i8.beam_select(dev(x) if isinstance(x, np.ndarray) else x, dev(scores),
                         None if live is None else dev(live),
                         eos=None if eos < 0 else eos, count=count, workspace=workspace)
    got = [host(o) for o in out]
    for name, g, w in zip(("tokens", "parents", "live"), got[1:], want[1:]):
        assert np.array_equal(g, w), name
    there = np.isfinite(want[0])
    assert np.array_equal(got[0][~there], want[0][~there].astype(np.float32))
    off = np.abs(got[0][there] - want[0][there])
    assert (off <= SUM + 2.0 ** -24 * np.abs(want[0][there])).all(), off.max()
    return got


def inputs(seed, batch, beams, vocab, half=True, spread=2.5, dead=True):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, spread, (batch, beams, vocab)).astype(np.float16 if half else np.float32)
    scores = (-6 * rng.random((batch, beams))).astype(np.float32)
    live = np.ones((batch, beams), np.int32)
    if dead:
        scores[rng.random(scores.shape) < 0.15] = -np.inf
        live[rng.random(live.shape) < 0.15] = 0
        x[rng.random(x.shape) < 0.05] = -np.inf
    return x, scores, live


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("batch,beams,vocab,count", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 2, 3), (1, 4, 63, 4), (3, 2, 64, 64), (2, 5, 65, 7),
    (1, 3, 1000, 64), (5, 7, 2047, 11), (1, 1, 8191, 1), (2, 2, 8193, 33), (4, 16, 4099, 32),
    (1, 64, 777, 64), (2, 6, 33000, 12), (1, 2, 70001, 17), (1, 300, 129, 20)])
def test_sizes(gpu, half, batch, beams, vocab, count):
    note("beam %s" % ((half, batch, beams, vocab, count),))
    x, scores, live = inputs(vocab + count, batch, beams, vocab, half)
    check(gpu, x, scores, live, eos=min(2, vocab - 1), count=count)


def test_many_rows_of_several_pieces(gpu):
    """More rows than blocks are wanted, each of more than one piece."""
    rng = np.random.default_rng(8)
    x = (rng.normal(0, 2.5, (130, 8, 66001))).astype(np.float16)
    scores = (-9 * rng.random((130, 8))).astype(np.float32)
    check(gpu, x, scores, None, eos=-1, count=8)


@pytest.mark.parametrize("half", [True, False])
def test_first_step_and_ended(gpu, half):
    """One beam to start from; all beams ended; no beam at all."""
    x, scores, live = inputs(1, 3, 4, 501, half, dead=False)
    scores[0, 1:] = -np.inf
    live[1] = 0
    scores[2] = -np.inf
    got = check(gpu, x, scores, live, count=4)
    assert (got[2][0] == 0).all()
    assert sorted(got[2][1]) == [4, 5, 6, 7] and (got[1][1] == 2).all() and (got[3][1] == 0).all()
    assert (got[2][2] == -1).all() and (got[1][2] == -1).all()


@pytest.mark.parametrize("half", [True, False])
def test_rows_without_candidates(gpu, half):
    """Rows of NaN, of +infinity, of -infinity only, scores that are not finite."""
    x, scores, live = inputs(2, 1, 8, 9000, half, dead=False)
    x[0, 0, 8999] = np.nan
    x[0, 1, 0] = np.inf
    x[0, 2] = -np.inf
    x[0, 3, 1:] = -np.inf
    scores[0, 4], scores[0, 5] = np.nan, np.inf
    x[0, 6] = np.nan      # not read: the beam has ended
    live[0, 6] = 0
    got = check(gpu, x, scores, live, count=16)
    assert set(got[2][0]) == {3, 6, 7}
    check(gpu, x[:, :3], scores[:, :3], live[:, :3].copy(), count=3)   # none at all


@pytest.mark.parametrize("half", [True, False])
def test_ties_go_to_the_lowest(gpu, half):
    """Constant rows, few distinct logits, equal beams, zeros of both signs."""
    kind = np.float16 if half else np.float32
    x = np.full((1, 3, 20000), 0.5, kind)
    got = check(gpu, x, np.zeros((1, 3), np.float32), None, eos=-1, count=10)
    assert got[1][0].tolist() == list(range(10)) and (got[2] == 0).all()
    rng = np.random.default_rng(4)
    x = rng.integers(0, 3, (2, 1, 30011)).astype(kind)
    check(gpu, x, np.zeros((2, 1), np.float32), None, eos=-1, count=64)
    x = np.zeros((1, 1, 5000), kind)
    x[0, 0, ::2] = -0.0
    got = check(gpu, x, np.zeros((1, 1), np.float32), None, eos=-1, count=5)
    assert got[1][0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("order", [1, -1])
def test_sorted_rows(gpu, order):
    """Every word beats the ones before it, or none does; most of the best in one
    lane's words."""
    x = np.linspace(-8, 8, 12345)[::order].astype(np.float32).reshape(1, 1, -1).copy()
    check(gpu, x, np.zeros((1, 1), np.float32), None, count=64)
    y = np.full((1, 1, 9000), -5.0, np.float16)
    y[0, 0, 800:808] = np.arange(8)[::order]
    y[0, 0, 2848:2856] = 10 + np.arange(8)[::order]
    check(gpu, y, np.zeros((1, 1), np.float32), None, eos=-1, count=30)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("count", [1, 64])
def test_long_pieces_of_many_good_words(gpu, half, count):
    """So many rows that a piece is all of one, of words that reach what has been seen
    before them: ascending, equal, of a few values; and the least that fp32 holds."""
    rng = np.random.default_rng(count)
    kinds = np.stack([np.linspace(-8, 8, 20001), np.linspace(8, -8, 20001), np.full(20001, -3.0),
                      rng.integers(0, 3, 20001), np.arange(20001) // 2500])
    if not half:
        kinds[2] = np.finfo(np.float32).min
        kinds[2, 50] = -np.inf
    x = np.tile(kinds.astype(np.float16 if half else np.float32), (210, 1)).reshape(1050, 1, -1)
    scores = (-6 * rng.random((1050, 1))).astype(np.float32)
    check(gpu, x, scores, None, eos=-1, count=count)


def test_no_beams_no_words(gpu):
    """Searches of no beams or no words: ended beams alone, or nothing."""
    for half in (np.float16, np.float32):
        got = check(gpu, np.zeros((2, 0, 50), half), np.zeros((2, 0), np.float32), None, count=3)
        assert (got[2] == -1).all()
        live = np.array([[0, 1, 0]], np.int32)
        got = check(gpu, np.zeros((1, 3, 0), half), np.array([[-2, 0, -1]], np.float32), live, eos=-1,
                    count=4)
        assert got[2].tolist() == [[2, 0, -1, -1]] and (got[1] == -1).all()
        many = -np.arange(300, dtype=np.float32)[None]
        got = check(gpu, np.zeros((1, 300, 0), half), many, np.zeros((1, 300), np.int32), eos=-1, count=5)
        assert got[2].tolist() == [[0, 1, 2, 3, 4]]
    assert gpu.beam_select(torch.zeros((0, 3, 9), device="cuda"),
                           torch.zeros((0, 3), device="cuda"))[0].shape == (0, 3)


@pytest.mark.parametrize("count", [1, 32, 64])
def test_joins_of_many_lists(gpu, count):
    """More entries than a join takes at once: many beams of many pieces, values of all
    beams close together and beams that lead by far."""
    rng = np.random.default_rng(count + 100)
    x = rng.normal(0, 2.5, (1, 40, 70000)).astype(np.float16)
    for spread in (0.0, 30.0):
        scores = (-spread * rng.random((1, 40))).astype(np.float32)
        check(gpu, x, scores, None, eos=-1, count=count)
    x = np.broadcast_to(rng.normal(0, 2.5, (1, 1, 30000)).astype(np.float16), (1, 40, 30000)).copy()
    check(gpu, x, np.zeros((1, 40), np.float32), None, eos=-1, count=count, equal_beams=True)


def test_large_and_small_logits(gpu):
    x = np.array([[[60000, 59968, -60000, 0], [-60000, -59968, -65504, -np.inf]]], np.float16)
    check(gpu, x, np.array([[-1.0, -2.0]], np.float32), None, eos=-1, count=4)
    y = np.array([[[3e38, -3e38, 2.9e38], [1e-40, 2e-40, 0]]], np.float32)
    got = gpu.beam_select(dev(y), dev(np.zeros((1, 2), np.float32)), count=4)
    assert host(got[1])[0, :1].tolist() == [0] and host(got[2])[0, :1].tolist() == [0]


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_alignment_and_strides(gpu, half, shift):
    """Rows that begin at any element, apart by more than their words; what lies
    between them is not taken."""
    x, scores, live = inputs(11 + shift, 3, 4, 2501, half)
    wide = torch.full((3 * 4 * 2600 + 16,), float("inf"), dtype=torch.float16 if half else torch.float32,
                      device="cuda")
    view = wide[shift:shift + 3 * 4 * 2600].view(3, 4, 2600)[:, :, :2501]
    view.copy_(dev(x))
    check(gpu, view, scores, live, count=9)


def test_rows_beyond_32_bit_offsets(gpu):
    """Rows more than 2^31 bytes apart."""
    x, scores, live = inputs(31, 1, 3, 5000, dead=False)
    wide = torch.empty((1, 3, (1 << 30) + 5000), dtype=torch.float16, device="cuda")[:, :, :5000]
    wide.copy_(dev(x))
    check(gpu, wide, scores, live, count=6)


def test_workspace_contents_do_not_matter(gpu):
    x, scores, live = inputs(21, 2, 3, 40000)
    need = gpu.load_library().i8mm_beam_select_workspace_bytes(0, 2, 3, 40000, 6)
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        check(gpu, x, scores, live, count=6, workspace=ws)
    asked = []

    def give(device, n):
        asked.append(n)
        return torch.full((n,), 255, dtype=torch.uint8, device=device)
    check(gpu, x, scores, live, count=6, workspace=give)
    assert asked == [need]
    with pytest.raises(gpu.I8mmError):
        gpu.beam_select(dev(x), dev(scores), dev(live), count=6, workspace=ws[:need - 1])


def test_recorded_and_on_another_stream(gpu):
    """Two recorded calls replayed with other inputs, eager ones in between."""
    x, scores, live = inputs(31, 2, 4, 30000)
    s = torch.cuda.Stream()
    gx, gs, gl = dev(x), dev(scores), dev(live)
    hx, hs, hl = gx.clone(), gs.clone(), gl.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gpu.beam_select(gx, gs, gl, eos=2)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = gpu.beam_select(gx, gs, gl, eos=2) + gpu.beam_select(hx, hs, hl, eos=2, count=9)
    for seed in (32, 33, 34):
        a, b = inputs(seed, 2, 4, 30000), inputs(seed + 50, 2, 4, 30000)
        for to, src in zip((gx, gs, gl, hx, hs, hl), a + b):
            to.copy_(dev(src))
        graph.replay()
        torch.cuda.synchronize()
        got = [host(o) for o in outs]
        for n, (inp, count) in enumerate(((a, 4), (b, 9))):
            eager = check(gpu, *inp, eos=2, count=count)
            for g, e in zip(got[4 * n:4 * n + 4], eager):
                assert np.array_equal(g, e)


def test_a_search_over_several_steps(gpu):
    """The outputs of a step are the inputs of the next."""
    rng = np.random.default_rng(40)
    scores = np.full((3, 4), -np.inf, np.float32)
    scores[:, 0] = 0
    live = np.ones((3, 4), np.int32)
    for _ in range(6):
        x = rng.normal(0, 3, (3, 4, 700)).astype(np.float16)
        x[:, :, 2] += 6
        got = check(gpu, x, scores, live, eos=2)
        scores, live = got[0], got[3]
    assert (live == 0).any()
