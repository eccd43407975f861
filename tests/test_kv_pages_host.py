"""Host-side checks of the calls on page tables: refusals of the C ABI and of the
binding (no GPU, no compute calls), and pins of the reference."""

import ctypes
import random

import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib, ops
from oracle import kv_pages as R

A, B, C = 0x100000, 0x200000, 0x300000   # aligned, never dereferenced
ODD = 0x10002     # not 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    return i8.ensure_built()


def call_step(lib, table=A, lens=A + 4096, seqs=3, width=5, parents=A, keep=None, new=None, new_all=1,
              rows=4, pages=20, page=64, out=B, out_lens=B + 4096, copies=C, counts=C + 4096, ws=A,
              wn=1 << 40):
    return lib.i8mm_kv_pages_step(table, lens, seqs, width, parents, keep, new, new_all, rows, pages,
                                  page, out, out_lens, copies, counts, ws, wn, None)


def call_compact(lib, table=A, lens=A, seqs=3, width=5, pages=20, page=64, out=B, copies=C, counts=C,
                 ws=A, wn=1 << 40):
    return lib.i8mm_kv_pages_compact(table, lens, seqs, width, pages, page, out, copies, counts, ws,
                                     wn, None)


def call_copy(lib, means=None, copies=A, count=A, most=4, **kw):
    f = dict(k_codes=A, k_absmax=A, v_codes=A, v_absmax=A, num_pages=8, page_tokens=64, kv_heads=2,
             head_dim=64)
    f.update(kw)
    return lib.int8_kv_cache_copy_pages(ctypes.byref(_lib.KVCacheStruct(**f)), means, copies, count,
                                        most, None)


BAD = [
    (dict(width=-1), _lib.I8MM_EINVAL), (dict(pages=-1), _lib.I8MM_EINVAL),
    (dict(seqs=-1), _lib.I8MM_EINVAL), (dict(seqs=65536), _lib.I8MM_EINVAL),
    (dict(page=0), _lib.I8MM_EINVAL), (dict(page=24), _lib.I8MM_EALIGN),
    (dict(page=1 << 17), _lib.I8MM_EINVAL), (dict(pages=1 << 31), _lib.I8MM_EINVAL),
    (dict(width=(1 << 24) + 1), _lib.I8MM_EINVAL), (dict(seqs=65535, width=1 << 15), _lib.I8MM_EINVAL),
    (dict(width=1 << 62), _lib.I8MM_EINVAL),
    (dict(table=None), _lib.I8MM_EINVAL), (dict(table=ODD), _lib.I8MM_EALIGN),
    (dict(lens=None), _lib.I8MM_EINVAL), (dict(lens=ODD), _lib.I8MM_EALIGN),
    (dict(out=None), _lib.I8MM_EINVAL), (dict(out=ODD), _lib.I8MM_EALIGN),
    (dict(out=A + 4), _lib.I8MM_EINVAL), (dict(copies=None), _lib.I8MM_EINVAL),
    (dict(counts=None), _lib.I8MM_EINVAL), (dict(counts=ODD), _lib.I8MM_EALIGN),
    (dict(ws=None, pages=20000), _lib.I8MM_EWORKSPACE), (dict(wn=79, pages=20000), _lib.I8MM_EWORKSPACE),
    (dict(ws=A + 16, pages=20000), _lib.I8MM_EALIGN)]


@pytest.mark.parametrize("kw,status", BAD)
def test_refused_by_both(lib, kw, status):
    assert call_step(lib, **kw) == status
    assert lib.i8mm_last_error().startswith(b"i8mm_kv_pages_step: ")
    assert call_compact(lib, **kw) == status
    assert lib.i8mm_last_error().startswith(b"i8mm_kv_pages_compact: ")


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), _lib.I8MM_EINVAL), (dict(rows=65536), _lib.I8MM_EINVAL),
    (dict(rows=65535, width=1 << 15), _lib.I8MM_EINVAL), (dict(new_all=-1), _lib.I8MM_EINVAL),
    (dict(new_all=1 << 31), _lib.I8MM_EINVAL), (dict(parents=None), _lib.I8MM_EINVAL),
    (dict(parents=ODD), _lib.I8MM_EALIGN), (dict(keep=ODD), _lib.I8MM_EALIGN),
    (dict(new=ODD), _lib.I8MM_EALIGN), (dict(out=A), _lib.I8MM_EINVAL),
    (dict(out_lens=None), _lib.I8MM_EINVAL), (dict(out_lens=A + 4096), _lib.I8MM_EINVAL),
    (dict(out=A - 4 * 19), _lib.I8MM_EINVAL)])
def test_refused_steps(lib, kw, status):
    assert call_step(lib, **kw) == status


def test_outputs_apart(lib):
    """No output overlaps another or an input, but for a compacted table that is the
    old one."""
    names = ("table", "lens", "parents", "keep", "new", "out", "out_lens", "copies", "counts")
    apart = {name: (2 + i) << 16 for i, name in enumerate(names)}
    for j, name in enumerate(names[5:], 5):
        for other in names[:j]:
            assert call_step(lib, **dict(apart, **{name: apart[other]})) == _lib.I8MM_EINVAL
            assert b"overlaps" in lib.i8mm_last_error()
    names = ("table", "lens", "out", "copies", "counts")
    apart = {name: apart[name] for name in names}
    for j, name in enumerate(names[2:], 2):
        for other in names[:j]:
            if (name, other) != ("out", "table"):
                assert call_compact(lib, **dict(apart, **{name: apart[other]})) == _lib.I8MM_EINVAL
                assert b"overlaps" in lib.i8mm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=-1), _lib.I8MM_EINVAL), (dict(page_tokens=24), _lib.I8MM_EALIGN),
    (dict(head_dim=72), _lib.I8MM_EINVAL), (dict(kv_heads=0), _lib.I8MM_EINVAL),
    (dict(k_codes=None), _lib.I8MM_EINVAL), (dict(v_absmax=A + 8), _lib.I8MM_EALIGN),
    (dict(means=A + 8), _lib.I8MM_EALIGN), (dict(most=-1), _lib.I8MM_EINVAL),
    (dict(most=1 << 31), _lib.I8MM_EINVAL), (dict(copies=None), _lib.I8MM_EINVAL),
    (dict(copies=ODD), _lib.I8MM_EALIGN), (dict(count=None), _lib.I8MM_EINVAL),
    (dict(count=ODD), _lib.I8MM_EALIGN)])
def test_refused_copies(lib, kw, status):
    assert call_copy(lib, **kw) == status
    assert lib.i8mm_last_error().startswith(b"int8_kv_cache_copy_pages: ")


def test_nothing_to_copy_needs_no_device(lib):
    assert lib.int8_kv_cache_copy_pages(None, None, A, A, 1, None) == _lib.I8MM_EINVAL
    assert call_copy(lib, most=0, copies=None, count=None) == _lib.I8MM_OK
    assert call_copy(lib, num_pages=0, k_codes=None, k_absmax=None, v_codes=None,
                     v_absmax=None) == _lib.I8MM_OK


def test_workspace_sizes(lib):
    """None for what one block does, room for a word, an entry and a place each beyond."""
    size = lib.i8mm_kv_pages_workspace_bytes
    assert size(-1, 4, 4) == size(4, -1, 4) == size(4, 4, -1) == size(65536, 4, 4) == 0
    assert size(0, 0, 1 << 31) == 0 and size(4, 17, 80) == 0
    for rows, width, pages in ((2000, 10, 100), (500, 1000, 100), (1, 1, 1 << 20), (65535, 100, 0)):
        assert size(rows, width, pages) >= 8 * (rows + pages)


def test_binding_refusals():
    t = torch.zeros((3, 5), dtype=torch.int32)
    n = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        ops.kv_pages_step(t.long(), n, n, 4, 64)
    with pytest.raises(TypeError):
        ops.kv_pages_step(t, n, [0, 1, 2], 4, 64)
    with pytest.raises(ValueError):
        ops.kv_pages_step(t, n[:2], n, 4, 64)
    with pytest.raises(ValueError):
        ops.kv_pages_step(t.T, n, n, 4, 64)
    with pytest.raises(ValueError):
        ops.kv_pages_step(t, n, n, 4, 64, new_tokens=n[:2])
    with pytest.raises(TypeError):
        ops.kv_pages_step(t, n, n, 4, 64, new_tokens=n.long())
    for keep in (n[:2], torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            ops.kv_pages_step(t, n, n, 4, 64, keep=keep)
    with pytest.raises(ValueError):                       # on the host
        ops.kv_pages_step(t, n, n, 4, 64)
    with pytest.raises(ValueError):
        ops.kv_pages_compact(t, n, 4, 64)
    with pytest.raises(ValueError):
        i8.KVPages(4, 24)
    with pytest.raises(ValueError):
        i8.KVPages(-1)


def test_reference_pins():
    """A search of two beams by hand, pages of 16 tokens."""
    table, lens = [[5, 1, -1], [5, 2, -1]], [20, 20]
    # both go on from beam 0: the first writes to its last page, the second to a copy
    out, n, copies, wanting = R.step(table, lens, [0, 0], [1, 1], None, 8, 16, 3)
    assert out == [[5, 1, -1], [5, 0, -1]] and n == [21, 21]
    assert copies == [(1, 0, 4)] and wanting == 0
    # one of them has ended, and keeps the page as it is
    out, _, copies, _ = R.step(table, lens, [0, 0], [1, 0], None, 8, 16, 3)
    assert out == [[5, 0, -1], [5, 1, -1]] and copies == [(1, 0, 4)]
    # a page that is full is shared; a new one begins
    out, n, copies, _ = R.step([[3, 4, -1]], [32], [0, 0, -1], [1, 1, 17], None, 8, 16, 3)
    assert out == [[3, 4, 0], [3, 4, 1], [2, 5, -1]] and n == [33, 33, 17] and not copies
    # cut back to 9 tokens; the pages run out
    out, n, copies, wanting = R.step([[0, 1, 2]], [40], [0, 0], [20, 20], [9, 30], 4, 16, 3)
    assert out == [[2, 3, -1], [0, 1, -1]] and n == [29, 48]
    assert copies == [(0, 2, 9)] and wanting == 1


def test_reference_properties():
    """No page is written by two rows, none that is read is given out."""
    rng = random.Random(2)
    for _ in range(200):
        page, width, pages = 16, 6, rng.randint(0, 30)
        rows = rng.randint(0, 6)
        table = [[rng.randint(-2, pages + 1) for _ in range(width)] for _ in range(rows)]
        lens = [rng.randint(-3, 110) for _ in range(rows)]
        count = rng.randint(0, 8)
        parents = [rng.randint(-1, rows) for _ in range(count)]
        new = [rng.randint(-1, 40) for _ in range(count)]
        keep = [rng.randint(-1, 100) for _ in range(count)] if rng.random() < 0.5 else None
        out, n, copies, wanting = R.step(table, lens, parents, new, keep, pages, page, width)
        targets = [c[1] for c in copies]
        assert len(set(targets)) == len(targets) and not set(targets) & {c[0] for c in copies}
        assert all(len(r) == width and all(-1 <= p < pages for p in r) for r in out)
        small, moves, live = R.compact(out, n, pages, page)
        assert all(p < live for r in small for p in r) and len(moves) <= pages // 2
        assert len({p for r in small for p in r if p >= 0}) == live
