"""Rows at the end of their page table, on the host: refusals of the step that gives the
batch's lengths too (no compute calls), and pins of the reference."""

import itertools
import random

import numpy as np
import pytest

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib
from oracle import kv_cache as C
from oracle import kv_pages as R
from tests.test_kv_cache_host import empty
from tests.test_kv_pages_host import BAD, ODD

NAMES = ("table", "lens", "parents", "keep", "new", "out", "out_lens", "batch_lens", "full", "copies",
         "counts")
APART = {name: (2 + i) << 16 for i, name in enumerate(NAMES)}   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return i8.ensure_built()


def call(lib, seqs=3, width=5, new_all=1, rows=4, pages=20, page=64, max_len=1 << 30, ws=1 << 24,
         wn=1 << 40, **kw):
    p = dict(APART, **kw)
    return lib.i8mm_kv_pages_step_batch(
        p["table"], p["lens"], seqs, width, p["parents"], p["keep"], p["new"], new_all, rows, pages, page,
        max_len, p["out"], p["out_lens"], p["batch_lens"], p["full"], p["copies"], p["counts"], ws, wn,
        None)


@pytest.mark.parametrize("kw,status", [b for b in BAD if "out" not in b[0] or b[0]["out"] != 0x100004] + [
    (dict(max_len=-1), _lib.I8MM_EINVAL), (dict(max_len=-1 << 63), _lib.I8MM_EINVAL),
    (dict(batch_lens=None), _lib.I8MM_EINVAL), (dict(batch_lens=ODD), _lib.I8MM_EALIGN),
    (dict(full=None), _lib.I8MM_EINVAL), (dict(full=ODD), _lib.I8MM_EALIGN),
    (dict(full=None, rows=0), _lib.I8MM_EINVAL)])
def test_refused(lib, kw, status):
    assert call(lib, **kw) == status
    assert lib.i8mm_last_error().startswith(b"i8mm_kv_pages_step_batch: ")


def test_outputs_apart(lib):
    for j, name in enumerate(NAMES[5:], 5):
        for other in NAMES[:j]:
            assert call(lib, **{name: APART[other]}) == _lib.I8MM_EINVAL
            assert b"overlaps" in lib.i8mm_last_error()


def test_sizes_at_their_extremes(lib):
    """In pairs, without the last output: every call is refused."""
    ends = (-1 << 63, -1, 0, 1, 15, 48, 1 << 20, 1 << 31, 1 << 40, 1 << 62, (1 << 63) - 1)
    names = ("seqs", "width", "rows", "pages", "page", "new_all", "max_len")
    for a, b in itertools.combinations(names, 2):
        for u, w in itertools.product(ends, ends):
            assert call(lib, counts=None, **{a: u, b: w}) < 0, (a, u, b, w)


def test_reference_pins():
    """Two beams go on from one whose table is full: its length does not grow, nothing
    is copied or wanting, and a batch of that length stores over its last token."""
    table, lens, copies, wanting = R.step([[0, 1]], [32], [0, 0], [1, 1], None, 10, 16, 2)
    assert table == [[0, 1], [0, 1]] and lens == [32, 32] and not copies and wanting == 0
    rng = np.random.default_rng(1)
    k, v = rng.normal(0, 1, (2, 32, 1, 64)).astype(np.float16)
    cache = empty(10, 1, 64, 16)
    C.append(cache, k, v, (np.array([[0, 1]]), [32], [32]))
    before = {name: x.copy() for name, x in cache.items()}
    C.append(cache, k[:2] * 3, v[:2] * 3, (np.array(table), lens, [1, 1]))
    assert not np.array_equal(cache["k_codes"][1], before["k_codes"][1])
    # of the lengths for a batch it stores nothing
    fed, full = R.batch_lens([32], [0, 0], [1, 1], None, 32)
    assert fed == [0, 0] and full == 2
    cache = {name: x.copy() for name, x in before.items()}
    C.append(cache, k[:2] * 3, v[:2] * 3, (np.array(table), fed, [1, 1]))
    assert all(np.array_equal(cache[name], before[name], equal_nan=True) for name in cache)
    # new tokens for some, room for some
    assert R.batch_lens([20, 32, 5], [0, 0, 1, 2, -1, 2], [12, 13, 1, 0, 33, 4], None, 32) == \
        ([32, 0, 0, 0, 0, 9], 3)
    assert R.batch_lens([40], [0, 0], [3, 3], [29, 30], 32) == ([32, 0], 1)
    assert R.step([[0, 1, 2]], [40], [0], [1], None, 10, 16, 3, max_len=40)[1] == [40]


def test_reference_lengths_agree():
    """A batch's length is the row's own, or 0; a row that is not full has all its tokens."""
    rng = random.Random(6)
    for _ in range(200):
        width, count = rng.randint(0, 4), rng.randint(0, 8)
        rows = rng.randint(0, 4)
        lens = [rng.randint(-3, 70) for _ in range(rows)]
        parents = [rng.randint(-1, rows) for _ in range(count)]
        new = [rng.randint(-1, 40) for _ in range(count)]
        limit = min(16 * width, rng.choice((1000, rng.randint(0, 64))))
        out = R.step([list(range(width))] * rows, lens, parents, new, None, 9, 16, width, max_len=limit)
        fed, full = R.batch_lens(lens, parents, new, None, limit)
        assert all(f in (0, n) for f, n in zip(fed, out[1])) and max(fed + [0]) <= limit
        assert full == sum(f == 0 and n > 0 for f, n in zip(fed, new))
