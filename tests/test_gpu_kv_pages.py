"""The calls on page tables and the copies of pages on the GPU against the plain
reference: every integer and every byte equal."""

import random

import numpy as np
import pytest
import torch

from oracle import kv_cache as C
from oracle import kv_pages as R
from tests.gpu_helpers import dev, host, note

pytestmark = pytest.mark.gpu


def ints(x, shape=None):
    a = np.array(x, np.int32)
    return dev(a if shape is None else a.reshape(shape))


def check_step(i8, table, lens, parents, new, keep, pages, page, width, pool=None):
    want = R.step(table, lens, parents, new if isinstance(new, list) else [new] * len(parents), keep,
                  pages, page, width)
    pool = pool or i8.KVPages(pages, page)
    t, n, copies = pool.step(ints(table, (len(table), width)), ints(lens, (len(table),)),
                             ints(parents, (len(parents),)),
                             ints(new, (len(parents),)) if isinstance(new, list) else new,
                             None if keep is None else ints(keep, (len(parents),)))
    assert host(t).tolist() == want[0]
    assert host(n).tolist() == want[1]
    rest = [[-1] * 3] * (len(parents) - len(want[2]))
    assert host(copies.pages).tolist() == [list(c) for c in want[2]] + rest
    assert host(copies.counts).tolist() == [len(want[2]), want[3]]
    return want, t, n, copies


def check_compact(i8, table, lens, pages, page, width):
    want = R.compact(table, lens, pages, page)
    t, copies = i8.KVPages(pages, page).compact(ints(table, (len(table), width)),
                                                ints(lens, (len(table),)))
    assert host(t).tolist() == want[0]
    rest = [[-1] * 3] * (pages // 2 - len(want[1]))
    assert host(copies.pages).tolist() == [list(c) for c in want[1]] + rest
    assert host(copies.counts).tolist() == [len(want[1]), want[2]]
    return want, t, copies


def random_rows(rng, rows, width, page, pages):
    """A table whose rows share some of their pages."""
    names = list(range(pages))
    rng.shuffle(names)
    table, lens, at = [], [], 0
    for i in range(rows):
        n = rng.randint(0, width)
        shared = rng.randint(0, n) if i and rng.random() < 0.5 else 0
        row = (table[rng.randrange(i)][:shared] if shared else [])
        row = [p for p in row if p >= 0]
        row = row + names[at:at + n - len(row)]
        at += n
        lens.append(max(0, len(row) * page - rng.choice((0, rng.randint(0, page - 1)))))
        table.append(row + [-1] * (width - len(row)))
    return table, lens


@pytest.mark.parametrize("rows,width,page,count", [
    (1, 1, 16, 1), (1, 3, 16, 5), (4, 5, 32, 4), (7, 300, 16, 9), (33, 17, 64, 64),
    (64, 129, 16, 200), (3, 9, 48, 1025), (300, 40, 16, 2100)])
@pytest.mark.parametrize("cut", [False, True])
def test_steps(gpu, rows, width, page, count, cut):
    rng = random.Random(rows * 1000 + width + cut)
    for room in (0, 3, 4 * count, 40 * count):
        table, lens = random_rows(rng, rows, width, page, rows * width)
        pages = 1 + max([p for r in table for p in r] + [0]) + room
        parents = [rng.randint(-1, rows) for _ in range(count)]
        new = [rng.choice((0, 1, 1, 1, rng.randint(0, 3 * page))) for _ in range(count)]
        keep = [rng.randint(0, width * page) for _ in range(count)] if cut else None
        note("step %s" % ((rows, width, page, count, cut, room),))
        check_step(gpu, table, lens, parents, new, keep, pages, page, width)


def test_one_number_of_new_tokens(gpu):
    table, lens = [[0, 1, -1, -1], [0, 2, -1, -1]], [20, 32]
    for n in (0, 1, 12, 13, 100):
        check_step(gpu, table, lens, [0, 0, 1, 1, -1], n, None, 12, 16, 4)
    with pytest.raises(gpu.I8mmError):
        gpu.KVPages(12, 16).step(ints(table), ints(lens), ints([0]), -1)


def test_what_the_arrays_hold_is_bounded(gpu):
    """Pages, parents, lengths and numbers of tokens that no user should pass."""
    big, low = 2 ** 31 - 1, -2 ** 31
    table = [[0, 1, 99, -5], [big, 2, 0, 0], [3, 3, 3, 3]]
    lens = [100, big, low]
    parents = [0, 1, 2, 3, -1, big, low, 0, 1]
    new = [1, big, 5, low, big, 1, 2, 0, -3]
    check_step(gpu, table, lens, parents, new, None, 40, 16, 4)
    check_step(gpu, table, lens, parents, new, [big, 17, low, 0, 1, 2, 3, 9, 33], 40, 16, 4)
    check_step(gpu, table, lens, parents, new, None, 0, 16, 4)       # no pages at all
    check_step(gpu, table, lens, [], 1, None, 40, 16, 4)             # every row ends
    check_step(gpu, [], [], [0, -1], 3, None, 40, 16, 2)             # nothing to begin with
    check_step(gpu, [[], []], [5, 0], [0, 1], 3, None, 40, 16, 0)    # no room in the table
    check_compact(gpu, table, lens, 40, 16, 4)
    check_compact(gpu, table, lens, 2, 16, 4)
    check_compact(gpu, table, lens, 0, 16, 4)
    check_compact(gpu, [], [], 9, 16, 0)


def test_a_long_prompt_and_many_pages(gpu):
    """One row that takes thousands of pages, out of tens of thousands."""
    table, lens = [[7, -1] + [-1] * 6000, [-1] * 6002], [20, 0]
    check_step(gpu, table, lens, [0, 0, 1, -1], [90000, 1, 0, 5000], None, 30000, 16, 6002)
    check_step(gpu, table, lens, [0, 0, 1, -1], [90000, 1, 0, 90000], None, 9000, 16, 6002)
    rng = random.Random(9)
    names = rng.sample(range(50000), 3000)
    check_compact(gpu, [names[:1500] + [-1] * 10, names[1490:]], [1500 * 16 - 3, 1510 * 16], 50000, 16,
                  1510)


@pytest.mark.parametrize("rows", [3, 70])
def test_rows_of_few_and_of_many_new_pages(gpu, rows):
    """Side by side, until the pages run out."""
    rng = np.random.default_rng(rows)
    new = [int(n) for n in rng.choice([0, 1, 17, 40, 100, 300, 4000], rows)]
    new[1] = 4700
    table, lens = rng.permutation(1500)[:10].reshape(1, 10), [150]
    table = np.concatenate([table, np.full((1, 290), -1)], axis=1).astype(np.int32)
    for pages in (20000, 1510, 1700):
        check_step(gpu, table, lens, [0] * rows, new, None, pages, 16, 300)


@pytest.mark.parametrize("rows,width,page", [(1, 1, 16), (3, 5, 32), (40, 300, 16), (300, 40, 64)])
def test_compact(gpu, rows, width, page):
    rng = random.Random(rows)
    for room in (0, 5, 3 * rows):
        table, lens = random_rows(rng, rows, width, page, rows * width + room)
        pages = rows * width + room
        (want, copies, live), t, _ = check_compact(gpu, table, lens, pages, page, width)
        # in place, and nothing more to do
        again = gpu.ops.kv_pages_compact(t, ints(lens), pages, page)
        assert host(again[0]).tolist() == want and host(again[2]).tolist() == [0, live]


def noise(rng, pages, heads, page, dim, means):
    shape = (pages, heads, page // 16)
    cache = {}
    for w in "kv":
        cache[w + "_codes"] = rng.integers(-127, 128, shape + (dim // 16, 16, 16)).astype(np.int8)
        cache[w + "_absmax"] = rng.random(shape).astype(np.float32)
    if means:
        cache["k_means"] = rng.normal(0, 1, (pages, heads, dim)).astype(np.float16)
    return cache


def gpu_cache(i8, cache):
    return i8.Int8KVCache.from_tensors(*(dev(cache[n]) for n in ("k_codes", "k_absmax", "v_codes",
                                                                 "v_absmax")),
                                       k_means=dev(cache["k_means"]) if "k_means" in cache else None)


def equal(c, cache):
    for name, x in cache.items():
        assert np.array_equal(host(getattr(c, name)), x), name


@pytest.mark.parametrize("heads,page,dim", [(1, 16, 64), (3, 48, 80), (2, 64, 96), (8, 64, 128),
                                            (5, 128, 256), (1, 2048, 64)])
@pytest.mark.parametrize("means", [False, True])
def test_copies(gpu, heads, page, dim, means):
    rng = np.random.default_rng(dim + heads)
    cache = noise(rng, 21, heads, page, dim, means)
    c = gpu_cache(gpu, cache)
    copies = [(0, 1, 1), (0, 2, 16), (0, 3, 17), (4, 5, page), (6, 7, 0), (8, 9, page - 1),
              (10, 10, page), (11, 21, page), (-1, 12, page), (13, -1, 5), (-1, -1, -1), (14, 15, -4),
              (16, 17, 2 ** 31 - 1), (18, 19, 5)]
    for count in (0, -7, 13, 14, 10 ** 6):
        note("copy %s" % ((heads, page, dim, count),))
        gpu.ops.int8_kv_cache_copy_pages(c, ints(copies), ints([count]))
        R.copy(cache, copies[:max(count, 0)], 21)
        equal(c, cache)


def test_many_copies(gpu):
    """More items than blocks are launched."""
    rng = np.random.default_rng(3)
    cache = noise(rng, 1200, 5, 16, 64, True)
    c = gpu_cache(gpu, cache)
    order = rng.permutation(1200)
    copies = [(int(order[2 * i]), int(order[2 * i + 1]), int(rng.integers(0, 17))) for i in range(600)]
    gpu.ops.int8_kv_cache_copy_pages(c, ints(copies), ints([600]))
    R.copy(cache, copies, 1200)
    equal(c, cache)


def test_copies_beyond_32_bit_offsets(gpu):
    """Pages whose bytes lie past 4 GiB."""
    pages, heads, page, dim = 4200, 32, 128, 256      # 1 MiB of keys a page
    c = gpu.Int8KVCache(pages, heads, dim, page)
    c.k_codes[0].fill_(5), c.v_codes[0].fill_(-6), c.k_absmax[0].fill_(2), c.v_absmax[0].fill_(3)
    c.k_codes[4199].zero_(), c.v_codes[4199].zero_(), c.k_absmax[4199].zero_(), c.v_absmax[4199].zero_()
    c.k_codes[4198].zero_(), c.v_codes[4198].zero_()
    gpu.ops.int8_kv_cache_copy_pages(c, ints([[0, 4199, 128]]), ints([1]))
    gpu.ops.int8_kv_cache_copy_pages(c, ints([[4199, 4198, 40]]), ints([1]))
    assert (c.k_codes[4199] == 5).all() and (c.v_codes[4199] == -6).all()
    assert (c.k_absmax[4199] == 2).all() and (c.v_absmax[4199] == 3).all()
    assert (c.k_codes[4198, :, :3] == 5).all() and (c.k_codes[4198, :, 3:] == 0).all()
    assert (c.v_codes[4198, :, :3] == -6).all() and (c.v_codes[4198, :, 3:] == 0).all()


def test_refused_tensors(gpu):
    c = gpu.Int8KVCache(4, 1, 64, 16)
    for pool in (gpu.KVPages(4, 32), gpu.KVPages(5, 16)):
        copies = pool.step(ints([[0]]), ints([9]), ints([0, 0]))[2]
        with pytest.raises(ValueError):
            c.copy_pages(copies)
    with pytest.raises(ValueError):
        gpu.ops.int8_kv_cache_copy_pages(c, ints([[0, 1]]), ints([1]))
    with pytest.raises(ValueError):
        gpu.ops.int8_kv_cache_copy_pages(c, torch.zeros((1, 3), dtype=torch.int32), ints([1]))
    with pytest.raises(TypeError):
        gpu.ops.int8_kv_cache_copy_pages(c, ints([[0, 1, 1]]), ints([1]).long())
    with pytest.raises(ValueError):
        gpu.Int8KVCache.from_tensors(c.k_codes, c.k_absmax, c.v_codes, c.v_absmax,
                                     k_means=torch.zeros((4, 1, 32), dtype=torch.float16, device="cuda"))


def test_workspace_contents_do_not_matter(gpu):
    table, lens, parents, pages = [[0, 1, 2], [0, 1, 19999]], [40, 47], [0, 0, 1, -1], 20000
    need = gpu.load_library().i8mm_kv_pages_workspace_bytes(4, 3, pages)
    want = R.step(table, lens, parents, [3] * 4, None, pages, 16, 3)
    assert need > 0
    for fill in (0, 255, 1, 128):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        t, n, copies, counts = gpu.ops.kv_pages_step(ints(table), ints(lens), ints(parents), pages, 16, 3,
                                                     workspace=ws)
        assert host(t).tolist() == want[0] and host(n).tolist() == want[1]
        ws.fill_(fill)
        t, _, _ = gpu.ops.kv_pages_compact(ints(table), ints(lens), pages, 16, workspace=ws)
        assert host(t).tolist() == R.compact(table, lens, pages, 16)[0]


@pytest.mark.parametrize("pages", [60, 17000])
def test_recorded_steps(gpu, pages):
    """A step, its copies and a compaction recorded once, replayed with other
    tables, with eager calls in between; in one launch each and in several."""
    rng = random.Random(5)
    nrng = np.random.default_rng(5)
    page, width, rows = 16, 6, 5
    pool = gpu.KVPages(pages, page)
    cache = noise(nrng, pages, 2, page, 64, True)
    c = gpu_cache(gpu, cache)
    table, lens, parents, new = (ints(np.zeros(s)) for s in ((rows, width), (rows,), (rows,), (rows,)))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c.copy_pages(pool.step(table, lens, parents, new)[2])
        c.copy_pages(pool.compact(table, lens)[1])
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t, n, copies = pool.step(table, lens, parents, new)
        c.copy_pages(copies)
        t2, copies2 = pool.compact(t, n)
        c.copy_pages(copies2)
    for x, name in ((c.k_codes, "k_codes"), (c.k_absmax, "k_absmax"), (c.v_codes, "v_codes"),
                    (c.v_absmax, "v_absmax"), (c.k_means, "k_means")):
        x.copy_(dev(cache[name]))
    for _ in range(4):
        rt, rl = random_rows(rng, rows, width, page, 25)
        rp = [rng.randint(-1, rows) for _ in range(rows)]
        rn = [rng.randint(0, 30) for _ in range(rows)]
        for to, src in ((table, rt), (lens, rl), (parents, rp), (new, rn)):
            to.copy_(ints(src))
        graph.replay()
        check_step(gpu, rt, rl, rp, rn, None, pages, page, width)
        wt, wl, wc, _ = R.step(rt, rl, rp, rn, None, pages, page, width)
        w2, wc2, _ = R.compact(wt, wl, pages, page)
        R.copy(cache, wc, pages)
        R.copy(cache, wc2, pages)
        assert host(t).tolist() == wt and host(n).tolist() == wl and host(t2).tolist() == w2
        equal(c, cache)


def test_a_search_over_a_cache(gpu):
    """Steps, copies and appends of a search whose beams part and end: the cache
    holds for every beam what its own tokens would have written alone."""
    rng = random.Random(11)
    nrng = np.random.default_rng(11)
    page, pages, width, heads, dim, beams = 32, 40, 4, 2, 64, 4
    pool = gpu.KVPages(pages, page)
    c = gpu.Int8KVCache(pages, heads, dim, page)
    for x in (c.k_codes, c.v_codes, c.k_absmax, c.v_absmax):
        x.zero_()
    table, lens = pool.empty_table(1, width * page)
    tokens = [[]]            # of each row: its (key, value) pairs
    parents, new = [-1], [40]
    for step in range(12):
        table, lens, copies = pool.step(table, lens, ints(parents), ints(new))
        c.copy_pages(copies)
        assert host(copies.counts)[1] == 0
        tokens = [list(tokens[p]) if p >= 0 else [] for p in parents]
        kv = nrng.normal(0, 1 + step % 3, (2, sum(new), heads, dim)).astype(np.float16)
        at = 0
        for row, n in zip(tokens, new):
            row += [(kv[0, at + i], kv[1, at + i], step) for i in range(n)]
            at += n
        cu = np.concatenate([[0], np.cumsum(new)])
        batch = gpu.KVBatch(table, lens, ints(cu), total_tokens=int(cu[-1]), max_tokens=max(new + [1]))
        c.append(dev(kv[0]), dev(kv[1]), batch)
        # each row's cache against appends of its own tokens alone, step by step
        for i, row in enumerate(tokens):
            alone = {n: np.zeros_like(host(getattr(c, n))[:width])
                     for n in ("k_codes", "v_codes", "k_absmax", "v_absmax")}
            line, done = np.arange(width)[None], 0
            for s in range(step + 1):
                part = [t for t in row if t[2] == s]
                if part:
                    done += len(part)
                    C.append(alone, np.stack([t[0] for t in part]), np.stack([t[1] for t in part]),
                             (line, [done], [len(part)]))
            ours = {n: host(getattr(c, n))[np.maximum(host(table)[i], 0)] for n in alone}
            want = C.read(alone, (line, [len(row)], [len(row)]))
            got = C.read(ours, (line, [len(row)], [len(row)]))
            assert len(row) == host(lens)[i]
            assert all(np.array_equal(a, b) for a, b in zip(got, want)), (step, i)
        rows = len(tokens)
        parents = [0] * beams if rows == 1 else [rng.choice((i, rng.randrange(rows), 0))
                                                 for i in range(beams)]
        new = [1] * beams if step < 7 else [rng.randint(0, 1) for _ in range(beams)]
