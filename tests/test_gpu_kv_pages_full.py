"""Rows that reach the end of their page table, or of the batches' max_len: the lengths
that a step gives for its append, and searches that grow past the end. Whole numbers and
cache bytes equal."""

import random

import numpy as np
import pytest
import torch

from oracle import kv_pages as R
from tests.gpu_helpers import dev, host, note
from tests.test_gpu_generation import Model, prompts
from tests.test_gpu_kv_pages import ints, random_rows

pytestmark = pytest.mark.gpu

NAMES = ("k_codes", "k_absmax", "v_codes", "v_absmax", "k_means")


@pytest.mark.parametrize("rows,width,page,count", [(1, 1, 16, 1), (4, 5, 32, 4), (7, 30, 16, 9),
                                                   (33, 2, 64, 64), (3, 9, 48, 1025), (300, 40, 16, 2100),
                                                   (2, 0, 16, 3), (0, 3, 16, 5)])
def test_lengths_for_the_batch(gpu, rows, width, page, count):
    """In one launch and in several, with tables and max_len that end in the new tokens."""
    rng = random.Random(rows * 100 + count)
    pool = gpu.KVPages(2 * rows * width + 40, page)
    for max_len in (None, 0, max(width * page - 5, 0), rng.randint(0, width * page), 1 << 40):
        for cut in (False, True):
            table, lens = random_rows(rng, rows, width, page, rows * width)
            lens = [rng.choice((n, width * page)) if -1 not in r else n for n, r in zip(lens, table)]
            parents = [rng.randint(-1, rows) for _ in range(count)]
            new = [rng.choice((-2, 0, 1, 1, rng.randint(0, 3 * page))) for _ in range(count)]
            keep = [rng.randint(0, width * page) for _ in range(count)] if cut else None
            note("full %s" % ((rows, width, page, count, max_len, cut),))
            want = R.step(table, lens, parents, new, keep, pool.num_pages, page, width, max_len)
            limit = width * page if max_len is None else min(width * page, max_len)
            fed, full = R.batch_lens(lens, parents, new, keep, limit)
            t, n, copies = pool.step(ints(table, (rows, width)), ints(lens, (rows,)), ints(parents),
                                     ints(new), None if keep is None else ints(keep), max_len=max_len)
            assert host(t).tolist() == want[0] and host(n).tolist() == want[1]
            assert host(copies.batch_lens).tolist() == fed and host(copies.full).tolist() == [full]
            assert host(copies.counts).tolist() == [len(want[2]), want[3]]
            assert host(copies.pages)[:len(want[2])].tolist() == [list(c) for c in want[2]]


def test_steps_of_one_number_of_new_tokens(gpu):
    pool = gpu.KVPages(12, 16)
    for n in (0, 1, 12, 13, 60):
        out = gpu.ops.kv_pages_step(ints([[0, 1, -1, -1]]), ints([20]), ints([0, 0, -1]), 12, 16, n,
                                    max_len=40, batch=True)
        fed, full = R.batch_lens([20], [0, 0, -1], [n] * 3, None, 40)
        assert host(out[4]).tolist() == fed and host(out[5]).tolist() == [full]
    assert pool.step(ints([[0]]), ints([9]), ints([]))[2].batch_lens.shape == (0,)
    with pytest.raises(gpu.I8mmError):
        pool.step(ints([[0]]), ints([9]), ints([0]), max_len=-1)


def test_full_rows_store_nothing(gpu):
    """Beams that share a full last page, one with room beside them: the step's own batch
    leaves every byte of the shared pages as it was."""
    rng = np.random.default_rng(3)
    page, heads = 16, 2
    pool = gpu.KVPages(8, page)
    c = gpu.Int8KVCache(8, heads, 64, page, page_means=True)
    for name in NAMES:
        getattr(c, name).zero_()
    table, lens = pool.empty_table(2, 32)
    table, lens, copies = pool.step(table, lens, ints([-1, -1]), ints([32, 20]))
    assert host(copies.batch_lens).tolist() == [32, 20] and host(copies.full).tolist() == [0]
    kv = dev(rng.normal(0, 1, (2, 52, heads, 64)).astype(np.float16))
    cu = ints([0, 32, 52])
    c.append(kv[0], kv[1], gpu.KVBatch(table, copies.batch_lens, cu, total_tokens=52, max_tokens=32))
    table, lens, copies = pool.step(table, lens, ints([0, 0, 1]))
    c.copy_pages(copies)
    assert host(copies.batch_lens).tolist() == [0, 0, 21] and host(copies.full).tolist() == [2]
    assert host(lens).tolist() == [32, 32, 21] and host(table)[0].tolist() == host(table)[1].tolist()
    before = {name: host(getattr(c, name)) for name in NAMES}
    batch = gpu.KVBatch(table, copies.batch_lens)
    q = dev(rng.normal(0, 1, (3, 4, 64)).astype(np.float16))
    c.append(*dev(rng.normal(0, 9, (2, 3, heads, 64)).astype(np.float16)), batch)
    changed = host(table)[2, 1]
    for name, x in before.items():
        now = host(getattr(c, name))
        assert np.array_equal(np.delete(now, changed, 0), np.delete(x, changed, 0)), name
    assert not np.array_equal(host(c.k_codes)[changed], before["k_codes"][changed])
    y = host(c.attention(q, batch))
    assert not y[:2].any() and y[2].any()


@pytest.mark.parametrize("limit,max_len", [(64, None), (64, 64), (64, 50)])
def test_a_search_past_the_end(gpu, limit, max_len):
    """Steps on after a search's beams are full: their pages keep every byte, the other
    search's beams are what they are alone, and `full` counts them."""
    rng = np.random.default_rng(7)
    model, page, beams = Model(gpu, rng), 16, 3
    end = max_len or limit
    pool = gpu.KVPages(60, page)
    caches = [gpu.Int8KVCache(60, 2, 64, page) for _ in range(2)]
    for c in caches:
        for name in NAMES[:4]:
            getattr(c, name).zero_()
    table, seq_lens, logits = prompts(gpu, model, rng, pool, caches, [end - 2, 7], limit)
    search = gpu.BeamSearch(pool, caches, table, seq_lens, beams, max_len=max_len)
    kept = None
    for step in range(6):
        note("past the end %s" % ((limit, max_len, step),))
        search.step(logits)
        assert int(search.full) == (0 if step < 2 else beams)
        assert host(search.seq_lens).tolist() == [min(end - 1 + step, end)] * beams + [8 + step] * beams
        fed = host(search.batch.seq_lens).tolist()
        assert fed == [end - 1 + step if step < 2 else 0] * beams + [8 + step] * beams
        x = model(torch.full((2 * beams,), 5 + step, device="cuda"), caches, search.batch)
        mine = [p for r in host(search.page_table)[:beams].tolist() for p in r if p >= 0]
        if step == 2:
            kept = mine, [{name: host(getattr(c, name)) for name in NAMES[:4]} for c in caches]
        if step > 2:
            for c, was in zip(caches, kept[1]):
                for name, before in was.items():
                    assert np.array_equal(host(getattr(c, name))[mine], before[mine]), (step, name)
        logits = model.head(x).view(2, beams, -1).clone()
        # (each beam goes on from itself)
        logits[0] = -30.0
        logits[0, :, step] = 30.0
