"""Attention over chosen pages of the 8-bit key/value cache on the GPU against the
numpy reference: mean keys and choices equal, attention within its derived bound."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as C
from oracle import kv_sparse as R
from tests.gpu_helpers import dev, host, note
from tests.test_gpu_kv_cache import make, on_gpu, tables

pytestmark = pytest.mark.gpu


def with_means(i8, rng, lens, counts, kv_heads, dim, page, cache=None, **kw):
    """A cache, its GPU form with mean keys of every page, and the batch."""
    cache, table = cache or make(rng, lens, kv_heads, dim, page)
    means = rng.normal(0, 1, (cache["k_absmax"].shape[0], kv_heads, dim)).astype(np.float16)
    R.page_means(cache, means, (table, lens, lens))
    c, b = on_gpu(i8, cache, table, lens, counts, max_len=max(lens), **kw)
    c = i8.Int8KVCache.from_tensors(c.k_codes, c.k_absmax, c.v_codes, c.v_absmax, k_means=dev(means))
    return cache, table, means, c, b


@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_means(gpu, dim, page):
    """Pages that begin and end anywhere among the new tokens; others stay."""
    rng = np.random.default_rng(dim + page)
    lens = [1, 16, 17, 130, 40, 95, 0, 300, 128]
    counts = [1, 1, 17, 130, 1, 60, 0, 3, 1]
    cache, table = make(rng, lens, 3, dim, page)
    table[4, 0] = -1
    table[5, 0] = 10 ** 6
    c, b = on_gpu(gpu, cache, table, lens, counts, max_len=300)
    means = rng.normal(0, 1, (cache["k_absmax"].shape[0], 3, dim)).astype(np.float16)
    c = gpu.Int8KVCache.from_tensors(c.k_codes, c.k_absmax, c.v_codes, c.v_absmax, k_means=dev(means))
    note("means %d %d" % (dim, page))
    for _ in range(2):
        c.update_means(b)
        R.page_means(cache, means, (table, lens, counts))
        assert np.array_equal(host(c.k_means), means)


def test_means_of_special_blocks(gpu):
    """A block of NaN, of infinities, of zeros; sums beyond fp16 become infinite."""
    rng = np.random.default_rng(1)
    cache, table = make(rng, [64, 64, 64, 64], 1, 64, 32, poison=False)
    for (b, j, s), a in zip(((0, 0, 0), (1, 1, 1), (2, 0, 1), (3, 0, 0)), (np.nan, np.inf, 0.0, 1e9)):
        cache["k_absmax"][table[b, j], :, s] = a
    cache["k_codes"][table[3, 0]] = 120
    means = np.zeros((cache["k_absmax"].shape[0], 1, 64), np.float16)
    c, b = on_gpu(gpu, cache, table, [64] * 4, [64] * 4)
    c = gpu.Int8KVCache.from_tensors(c.k_codes, c.k_absmax, c.v_codes, c.v_absmax, k_means=dev(means))
    c.update_means(b)
    R.page_means(cache, means, (table, [64] * 4, [64] * 4))
    assert np.array_equal(host(c.k_means), means, equal_nan=True)


def check_select(i8, rng, lens, counts, heads, kv_heads, dim, page, count, first=1, recent=1, rotary=0,
                 interleaved=False, q=None, prepared=None, **kw):
    cache, table, means, c, b = prepared or with_means(i8, rng, lens, counts, kv_heads, dim, page, **kw)
    if q is None:
        q = rng.normal(0, 1.5, (sum(counts), heads, dim)).astype(np.float16)
    cos = sin = rot = None
    if rotary:
        cos, sin = tables(rotary, max(lens) + 1)
        rot = i8.Rotary(dev(cos), dev(sin), interleaved)
    got = host(c.select_pages(dev(q), b, count, rot, first, recent))
    want, gap = R.select_pages(cache, means, q, (table, lens, counts), count, first, recent, cos, sin,
                               interleaved)
    # both sides' 64-bit sums of up to 2^12 products are off by less
    assert gap > 1e-9, gap
    assert np.array_equal(got, want)
    return got


@pytest.mark.parametrize("dim,rotary,interleaved", [
    (64, 0, False), (64, 64, True), (80, 80, False), (96, 32, False), (128, 128, False), (128, 64, True),
    (256, 256, False), (256, 0, False)])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_select(gpu, dim, rotary, interleaved, group):
    """Tokens with fewer, as many and more pages than are chosen."""
    rng = np.random.default_rng(dim + group)
    note("select %s" % ((dim, rotary, interleaved, group),))
    lens, counts = [1, 700, 63, 64, 65, 400, 0, 17], [1, 2, 63, 1, 20, 1, 0, 1]
    check_select(gpu, rng, lens, counts, 2 * group, 2, dim, 16, 4, rotary=rotary, interleaved=interleaved)
    check_select(gpu, rng, lens, counts, 2 * group, 2, dim, 32, 7, first=2, recent=3, rotary=rotary,
                 interleaved=interleaved)


def test_select_counts(gpu):
    """No page by its score, one, all but one; none of the first."""
    rng = np.random.default_rng(3)
    lens, counts = [333, 90], [3, 1]
    prepared = with_means(gpu, rng, lens, counts, 1, 64, 16)
    for count, first, recent in ((1, 0, 1), (2, 1, 1), (2, 0, 1), (20, 1, 1), (20, 0, 1), (21, 1, 1),
                                 (22, 1, 1), (100, 1, 1), (9, 4, 5), (10, 4, 5), (6, 0, 6)):
        check_select(gpu, rng, lens, counts, 2, 1, 64, 16, count, first, recent, prepared=prepared)


def test_select_many_pages(gpu):
    """More pages than one round of a block takes, than a block of 256 is given."""
    rng = np.random.default_rng(4)
    for pages, count in ((517, 100), (1500, 700), (2100, 17)):
        check_select(gpu, rng, [16 * pages - 5], [2], 4, 2, 64, 16, count, first=1, recent=2)


def test_select_many_blocks(gpu):
    """The same for more blocks than compute units."""
    rng = np.random.default_rng(41)
    check_select(gpu, rng, [16 * 600 - 5], [40], 8, 8, 64, 16, 33, first=1, recent=2)


def test_select_the_most_pages(gpu):
    """As many candidates as are allowed; the reference is torch's sort."""
    pages, kv_heads, dim, count = 16386, 1, 64, 50
    means = torch.randn((pages, kv_heads, dim), device="cuda").half()
    codes = torch.zeros((pages, 1, 1, 4, 16, 16), dtype=torch.int8, device="cuda")
    absmax = torch.ones((pages, 1, 1), device="cuda")
    c = gpu.Int8KVCache.from_tensors(codes, absmax, codes, absmax, k_means=means)
    order = torch.randperm(pages, device="cuda").int()
    b = gpu.KVBatch(order[None].contiguous(), torch.tensor([pages * 16], dtype=torch.int32, device="cuda"))
    q = torch.randn((1, 2, dim), device="cuda").half()
    got = c.select_pages(q, b, count)[0, 0].long()
    score = means[order.long(), 0].double() @ q[0].double().sum(dim=0)
    score[0] = score[-1] = float("inf")
    assert got.tolist() == torch.sort(score, descending=True, stable=True)[1][:count].sort()[0].tolist()
    b = gpu.KVBatch(torch.zeros((1, 16387), dtype=torch.int32, device="cuda"), b.seq_lens)
    with pytest.raises(gpu.I8mmError):
        c.select_pages(q, b, count)


def test_select_ties_nan_and_absent(gpu):
    """Equal means go by number; pages absent, of NaN means and infinite scores."""
    rng = np.random.default_rng(5)
    lens, counts = [640, 640], [1, 4]
    cache, table = make(rng, lens, 1, 64, 16)
    for prepare in ("equal", "few", "special"):
        means = np.ones((cache["k_absmax"].shape[0], 1, 64), np.float16)
        tab = table.copy()
        if prepare == "few":
            means[:] = rng.integers(0, 3, (means.shape[0], 1, 1))
        if prepare == "special":
            means = rng.normal(0, 1, means.shape).astype(np.float16)
            means[table[0, 3:9]] = np.nan
            means[table[0, 11]] = np.inf
            means[table[1, 5], 0, 0], means[table[1, 6], 0, 1] = np.inf, -np.inf
            tab[0, 15], tab[1, 20], tab[1, 38] = -1, 10 ** 9, -7
        c, b = on_gpu(gpu, cache, tab, lens, counts, max_len=640)
        c = gpu.Int8KVCache.from_tensors(c.k_codes, c.k_absmax, c.v_codes, c.v_absmax, k_means=dev(means))
        for count in (5, 36, 39):
            check_select(gpu, rng, lens, counts, 2, 1, 64, 16, count, first=1, recent=1,
                         q=np.ones((5, 2, 64), np.float16), prepared=(cache, tab, means, c, b))
    q = rng.normal(0, 1, (5, 2, 64)).astype(np.float16)
    q[0, 0, 3], q[1, 1, 7], q[2, 0, 1], q[2, 1, 1] = np.nan, np.inf, np.inf, -np.inf
    check_select(gpu, rng, lens, counts, 2, 1, 64, 16, 7, q=q, prepared=(cache, tab, means, c, b))


def chosen_for(rng, lens, counts, kv_heads, page, count, junk=False):
    """Lists of pages: some a token sees, in order or not, some it does not."""
    out = np.full((sum(counts), kv_heads, count), -1, np.int32)
    row = 0
    for l, n in zip(lens, counts):
        for i in range(n):
            seen = max(l - n + i, 0) // page + 1
            for h in range(kv_heads):
                if junk:
                    out[row, h] = rng.integers(-3, seen + 3, count)
                    out[row, h, rng.random(count) < 0.1] = 2 ** 31 - 1
                    continue
                k = min(seen, count, int(rng.integers(1, count + 1)))
                out[row, h, :k] = np.sort(rng.permutation(seen)[:k])
            row += 1
    return out


def check_attention(i8, rng, lens, counts, heads, kv_heads, dim, page, count, rotary=0, interleaved=False,
                    junk=False, chosen=None, cache=None, q=None, scale=None, max_len=None):
    cache, table = cache or make(rng, lens, kv_heads, dim, page)
    if q is None:
        q = rng.normal(0, 1.5, (sum(counts), heads, dim)).astype(np.float16)
    cos = sin = rot = None
    if rotary:
        cos, sin = tables(rotary, max(lens) + 1)
        rot = i8.Rotary(dev(cos), dev(sin), interleaved)
    c, b = on_gpu(i8, cache, table, lens, counts, max_len=max(lens) if max_len is None else max_len)
    if chosen is None:
        chosen = chosen_for(rng, lens, counts, kv_heads, page, count, junk)
    got = host(c.attention_pages(dev(q), dev(chosen), b, rot, scale=scale)).astype(np.float64)
    want, bound = R.attention_pages(cache, q, (table, lens, counts), chosen, cos, sin, interleaved, scale)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / bound) if got.size else 0.0
    assert worst <= 1.0, worst
    return got


@pytest.mark.parametrize("dim,rotary,interleaved", [
    (64, 0, False), (64, 32, True), (80, 80, False), (96, 96, False), (128, 128, False), (128, 64, True),
    (256, 0, False), (256, 256, True)])
@pytest.mark.parametrize("page,count", [(16, 5), (48, 3), (128, 2)])
def test_attention(gpu, dim, rotary, interleaved, page, count):
    rng = np.random.default_rng(dim + page)
    note("attention over pages %s" % ((dim, rotary, interleaved, page, count),))
    check_attention(gpu, rng, [1, 300, 47, 49, 129, 0, 17], [1, 3, 5, 1, 1, 0, 17], 4, 2, dim, page, count,
                    rotary, interleaved)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (16, 2), (17, 1), (33, 1), (40, 1), (24, 3),
                                            (7, 1), (9, 1)])
def test_shared_heads(gpu, heads, kv_heads):
    """Groups of one head, of a tile, of several tiles."""
    rng = np.random.default_rng(heads)
    check_attention(gpu, rng, [200, 33], [2, 1], heads, kv_heads, 64, 16, 6, 64)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_lists_of_any_kind(gpu, dim):
    """Unordered, repeated, negative and unseen pages, absent ones, empty lists."""
    rng = np.random.default_rng(dim)
    for count in (1, 7, 70):
        check_attention(gpu, rng, [500, 64, 15, 1], [9, 2, 15, 1], 4, 2, dim, 16, count, junk=True)
    cache, table = make(rng, [300, 300], 2, dim, 16)
    table[0, 3], table[1, 0], table[1, 18] = -1, 10 ** 8, -9
    check_attention(gpu, rng, [300, 300], [2, 2], 4, 2, dim, 16, 12, junk=True, cache=(cache, table))
    none = np.full((4, 2, 3), -1, np.int32)
    got = check_attention(gpu, rng, [300, 300], [2, 2], 4, 2, dim, 16, 3, chosen=none, cache=(cache, table))
    assert not got.any()


@pytest.mark.parametrize("dim", [64, 128])
def test_lists_longer_than_their_sequence(gpu, dim):
    """Pages listed many times: the last split of a list takes what is left of it."""
    rng = np.random.default_rng(dim + 5)
    chosen = rng.integers(-2, 40, (3, 2, 200)).astype(np.int32)
    chosen[1, 0, 30:] = -1
    check_attention(gpu, rng, [600, 40], [2, 1], 6, 2, dim, 16, 200, chosen=chosen)


@pytest.mark.parametrize("dim,rotary,interleaved", [
    (64, 64, False), (80, 0, False), (96, 96, True), (128, 64, False), (256, 256, False)])
@pytest.mark.parametrize("group", [1, 3, 4, 5, 8])
def test_many_tokens(gpu, dim, rotary, interleaved, group):
    """Enough tokens for a wave each: chunks and single tokens, lists longer than the
    wave's list of blocks and lists that end inside a set of groups."""
    rng = np.random.default_rng(dim + group)
    note("many tokens %s" % ((dim, rotary, interleaved, group),))
    lens, counts = [190, 1, 150, 0, 40, 301], [150, 1, 131, 0, 37, 6]
    check_attention(gpu, rng, lens, counts, 8 * group, 8, dim, 16, 7, rotary, interleaved)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [2, 7])
def test_many_tokens_lists_of_any_kind(gpu, dim, group):
    rng = np.random.default_rng(dim + group)
    lens, counts = [1300, 270, 9], [3, 80, 3]
    cache, table = make(rng, lens, 32, dim, 48)
    table[0, 3], table[1, 2] = -1, 10 ** 9
    check_attention(gpu, rng, lens, counts, 32 * group, 32, dim, 48, 30, junk=True, cache=(cache, table))
    none = np.full((86, 32, 2), -1, np.int32)
    got = check_attention(gpu, rng, lens, counts, 32 * group, 32, dim, 48, 2, chosen=none,
                          cache=(cache, table))
    assert not got.any()


def test_many_tokens_some_of_no_sequence(gpu):
    """Rows past the sequences, beyond max_tokens, before a sequence; special queries."""
    rng = np.random.default_rng(22)
    lens, counts, heads, kv = [100, 3], [40, 30], 64, 32
    cache, table = make(rng, lens, kv, 64, 16, poison=False)
    c, _ = on_gpu(gpu, cache, table, lens, counts)
    cu = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    b = gpu.KVBatch(dev(table), dev(np.array(lens, np.int32)), cu, total_tokens=90, max_tokens=35,
                    max_len=100)
    q = rng.normal(0, 1, (90, heads, 64)).astype(np.float16)
    q[3, 5, 7], q[4, 6, 8] = np.nan, np.inf
    cos, sin = tables(64, 100)
    chosen = np.sort(rng.integers(-1, 7, (90, kv, 4)).astype(np.int32), axis=2)
    out = torch.full((90, heads, 64), float("nan"), dtype=torch.float16, device="cuda")
    c.attention_pages(dev(q), dev(chosen), b, gpu.Rotary(dev(cos), dev(sin)), out=out)
    got = host(out).astype(np.float64)
    assert np.isnan(got[3, 5]).all() and np.isnan(got[4, 6]).all()
    q[3, 5], q[4, 6] = 0, 0
    got[3, 5] = got[4, 6] = 0
    # the first sequence's rows are tokens 65 .. 99 of 35, the second's -27 .. 2 of 30
    want, bound = R.attention_pages(cache, q[:35], (table, [100], [35]), chosen[:35], cos, sin)
    want[3, 5] = want[4, 6] = 0
    assert (np.abs(got[:35] - want) <= bound).all()
    assert not got[35:67].any() and not got[70:].any()
    want, bound = R.attention_pages(cache, q[67:70], (table[1:], [3], [3]), chosen[67:70], cos, sin)
    assert (np.abs(got[67:70] - want) <= bound).all()


def test_both_kernels_agree(gpu):
    """The same tokens alone and among many: each within its bound of the reference, so
    within both of each other."""
    rng = np.random.default_rng(23)
    lens, counts = [400] * 3, [100] * 3
    cache, table = make(rng, lens, 16, 64, 16)
    q = rng.normal(0, 1.5, (300, 64, 64)).astype(np.float16)
    chosen = chosen_for(rng, lens, counts, 16, 16, 9)
    c, b = on_gpu(gpu, cache, table, lens, counts, max_len=400)
    many = host(c.attention_pages(dev(q), dev(chosen), b)).astype(np.float64)
    last = [99, 199, 299]
    one = gpu.KVBatch(b.page_table, b.seq_lens, max_len=400)
    few = host(c.attention_pages(dev(q[last]), dev(chosen[last]), one)).astype(np.float64)
    _, bound = R.attention_pages(cache, q[last], (table, lens, [1] * 3), chosen[last])
    assert (np.abs(many[last] - few) <= 2 * bound).all()


def test_long_lists_are_split(gpu):
    """Lists of many splits, and of more than the joins of few take."""
    rng = np.random.default_rng(9)
    for tokens, count, heads, kv in ((2100, 130, 2, 1), (9000, 560, 4, 2), (600, 40, 8, 1)):
        check_attention(gpu, rng, [tokens, 40], [1, 1], heads, kv, 64, 16, count)


def test_every_page_equals_the_dense_attention(gpu):
    """All pages in order: the dense call's result, within both bounds (the dense
    call's for few rows)."""
    rng = np.random.default_rng(10)
    lens, counts = [777, 64, 30], [1, 1, 1]
    cache, table = make(rng, lens, 2, 128, 32)
    q = rng.normal(0, 1.5, (3, 8, 128)).astype(np.float16)
    chosen = np.broadcast_to(np.arange(25, dtype=np.int32), (3, 2, 25)).copy()
    got = check_attention(gpu, rng, lens, counts, 8, 2, 128, 32, 25, chosen=chosen, cache=(cache, table), q=q)
    c, b = on_gpu(gpu, cache, table, lens, counts, max_len=777)
    dense = host(c.attention(dev(q), b)).astype(np.float64)
    _, bound = C.attention(cache, q, (table, lens, counts))
    assert (np.abs(got - dense) <= 2 * bound).all()


def test_beyond_32_bit_offsets(gpu):
    """Pages past 2^31 bytes of codes: as the same pages at the front of a small cache."""
    rng = np.random.default_rng(77)
    pages, n, dim, kv, page = 34000, 12, 128, 8, 64
    small = gpu.Int8KVCache(n, kv, dim, page, page_means=True)
    big = gpu.Int8KVCache(pages, kv, dim, page, page_means=True)
    order = rng.permutation(n)
    table = torch.from_numpy(order.reshape(1, n).astype(np.int32)).cuda()
    lens = torch.tensor([n * page - 5], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n * page - 5], dtype=torch.int32, device="cuda")
    k, v = (dev(rng.normal(0, 1, (n * page - 5, kv, dim)).astype(np.float16)) for _ in range(2))
    q = dev(rng.normal(0, 1.5, (1, 4 * kv, dim)).astype(np.float16))
    found = []
    for cache, shift in ((small, 0), (big, pages - n)):
        cache.append(k, v, gpu.KVBatch(table + shift, lens, cu, n * page - 5, n * page - 5))
        one = gpu.KVBatch(table + shift, lens)
        chosen = cache.select_pages(q, one, 5, first=1, recent=2)
        found.append((cache.k_means[shift:shift + n].clone(), chosen, cache.attention_pages(q, chosen, one)))
    for a, b in zip(*found):
        assert torch.equal(a, b)
    assert found[0][2].abs().sum() > 0


def test_rows_of_no_sequence(gpu):
    """Rows past the last sequence, tokens beyond max_tokens and at negative
    positions: 0, and a choice of -1."""
    rng = np.random.default_rng(12)
    lens, counts = [100, 2], [2, 5]
    cache, table, means, c, b = with_means(gpu, rng, lens, counts, 2, 64, 16)
    cu = torch.tensor([0, 2, 7], dtype=torch.int32, device="cuda")
    b = gpu.KVBatch(b.page_table, b.seq_lens, cu, total_tokens=11, max_tokens=4, max_len=100)
    q = rng.normal(0, 1, (11, 4, 64)).astype(np.float16)
    cos, sin = tables(64, 100)
    rot = gpu.Rotary(dev(cos), dev(sin))
    picked = c.select_pages(dev(q), b, 3, rot)
    want, _ = R.select_pages(cache, means, q[:2], (table, lens[:1], [2]), 3, cos=cos, sin=sin)
    assert np.array_equal(host(picked)[:2], want)
    # the second sequence's four rows are its last: positions -2 .. 1
    assert (host(picked)[2:4] == -1).all() and (host(picked)[6:] == -1).all()
    assert (host(picked)[4:6] == [0, -1, -1]).all()
    out = torch.full((11, 4, 64), float("nan"), dtype=torch.float16, device="cuda")
    c.attention_pages(dev(q), torch.zeros_like(picked), b, rot, out=out)
    got = host(out).astype(np.float64)
    assert not got[2:4].any() and not got[6:].any() and np.isfinite(got).all()
    ref, bound = R.attention_pages(cache, q[:2], (table, lens[:1], [2]), np.zeros((2, 2, 3), int), cos, sin)
    assert (np.abs(got[:2] - ref) <= bound).all()
    ref, bound = R.attention_pages(cache, q[4:6], (table[1:], [2], [2]), np.zeros((2, 2, 3), int), cos, sin)
    assert (np.abs(got[4:6] - ref) <= bound).all()
    empty = gpu.KVBatch(b.page_table, torch.zeros_like(b.seq_lens), torch.zeros_like(cu), total_tokens=11,
                        max_tokens=4, max_len=100)
    assert (host(c.select_pages(dev(q), empty, 3, rot)) == -1).all()
    assert not host(c.attention_pages(dev(q), picked, empty, rot)).any()
    nowhere = gpu.KVBatch(b.page_table, b.seq_lens, cu, total_tokens=11, max_tokens=0, max_len=100)
    assert (host(c.select_pages(dev(q), nowhere, 3, rot)) == -1).all()
    assert not host(c.attention_pages(dev(q), picked, nowhere, rot)).any()
    c.update_means(nowhere)
    c.update_means(empty)
    assert np.array_equal(host(c.k_means), means)


def test_no_tokens_no_pages(gpu):
    c = gpu.Int8KVCache(0, 2, 64, 16, page_means=True)
    table = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    b = gpu.KVBatch(table, torch.tensor([40, 9], dtype=torch.int32, device="cuda"))
    q = torch.ones((2, 4, 64), dtype=torch.float16, device="cuda")
    c.update_means(b)
    assert (host(c.select_pages(q, b, 2)) == -1).all()
    assert not host(c.attention_pages(q, torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda"), b)).any()
    b = gpu.KVBatch(table[:0], b.seq_lens[:0])
    assert c.select_pages(q[:0], b, 2).shape == (0, 2, 2)
    assert c.attention_pages(q[:0], torch.zeros((0, 2, 3), dtype=torch.int32, device="cuda"), b).shape \
        == (0, 4, 64)


def test_many_sequences(gpu):
    """More sequences than a wave has lanes, empty ones among them."""
    rng = np.random.default_rng(14)
    counts = [int(x) for x in rng.integers(0, 4, 300)]
    lens = [n + int(rng.integers(0, 60)) if n else int(rng.integers(0, 50)) for n in counts]
    check_attention(gpu, rng, lens, counts, 2, 1, 64, 16, 3, 64)
    check_select(gpu, rng, lens, counts, 2, 1, 64, 16, 2, first=0, rotary=64)


def test_special_queries(gpu):
    """A NaN or an infinity in a query gives NaN for its own head; weights that
    underflow, large scores."""
    rng = np.random.default_rng(15)
    cache, table = make(rng, [200], 1, 64, 16, poison=False)
    q = rng.normal(0, 1.5, (1, 4, 64)).astype(np.float16)
    q[0, 1, 5], q[0, 2, 9] = np.nan, -np.inf
    c, b = on_gpu(gpu, cache, table, [200], [1], max_len=200)
    chosen = np.array([[[0, 3, 12]]], np.int32)
    got = host(c.attention_pages(dev(q), dev(chosen), b))
    assert np.isnan(got[0, 1:3]).all() and np.isfinite(got[0, [0, 3]]).all()
    check_attention(gpu, rng, [200], [1], 4, 1, 64, 16, 3, chosen=chosen, cache=(cache, table),
                    q=np.full((1, 4, 64), 30, np.float16), scale=4.0)
    check_attention(gpu, rng, [200], [1], 4, 1, 64, 16, 3, chosen=chosen, cache=(cache, table),
                    q=np.zeros((1, 4, 64), np.float16))


def test_strides_and_shared_prefixes(gpu):
    """Queries that are slices of a fused projection; two sequences on one page."""
    rng = np.random.default_rng(16)
    cache, table = make(rng, [90, 90], 2, 64, 16)
    table[1, :4] = table[0, :4]
    fused = rng.normal(0, 1, (2, 8, 64)).astype(np.float16)
    chosen = np.array([[[0, 2, 5], [1, 3, -1]]] * 2, np.int32)
    c, b = on_gpu(gpu, cache, table, [90, 90], [1, 1], max_len=90)
    got = host(c.attention_pages(dev(fused)[:, 2:6], dev(chosen), b)).astype(np.float64)
    want, bound = R.attention_pages(cache, fused[:, 2:6], (table, [90, 90], [1, 1]), chosen)
    assert (np.abs(got - want) <= bound).all()


def test_workspace_contents_do_not_matter(gpu):
    rng = np.random.default_rng(17)
    cache, table = make(rng, [4000], 1, 64, 16)
    c, b = on_gpu(gpu, cache, table, [4000], [1], max_len=4000)
    q = rng.normal(0, 1.5, (1, 2, 64)).astype(np.float16)
    chosen = np.sort(rng.permutation(250)[:100]).astype(np.int32).reshape(1, 1, 100)
    need = gpu.load_library().int8_kv_cache_attention_pages_workspace_bytes(c.ref, b.ref, 2, 100)
    assert need > 0
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        outs.append(host(gpu.ops.int8_kv_cache_attention_pages(dev(q), dev(chosen), c, b, workspace=ws)))
    want, bound = R.attention_pages(cache, q, (table, [4000], [1]), chosen)
    assert (np.abs(outs[0] - want) <= bound).all()
    assert all(np.array_equal(o, outs[0]) for o in outs)


def test_recorded_step(gpu):
    """Append, means, choice and attention recorded once and replayed while the
    sequences grow, against the eager calls."""
    rng = np.random.default_rng(18)
    lens = [70, 200, 33]
    cache, table, means, c, b = with_means(gpu, rng, lens, [1] * 3, 2, 64, 16)
    table = dev(np.concatenate([table, np.full((3, 2), -1, np.int32)], axis=1))
    used = set(host(table).ravel().tolist())
    spare = [p for p in range(cache["k_absmax"].shape[0]) if p not in used]
    table[2, 3] = spare[0]
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    batch = gpu.KVBatch(table, seq_lens, max_len=256)
    cos, sin = tables(64, 256)
    rot = gpu.Rotary(dev(cos), dev(sin))
    k, v = (torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")

    def step(c):
        c.append(k, v, batch, rot)
        c.update_means(batch)
        pages = c.select_pages(q, batch, 4, rot)
        return pages, c.attention_pages(q, pages, batch, rot)

    twin = gpu.Int8KVCache.from_tensors(*(getattr(c, n).clone() for n in (
        "k_codes", "k_absmax", "v_codes", "v_absmax", "k_means")))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(gpu.Int8KVCache.from_tensors(*(getattr(c, n).clone() for n in (
            "k_codes", "k_absmax", "v_codes", "v_absmax", "k_means"))))
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pages, out = step(c)
    for _ in range(5):
        for x in (k, v, q):
            x.copy_(dev(rng.normal(0, 1, x.shape).astype(np.float16)))
        seq_lens += 1
        graph.replay()
        want = step(twin)
        torch.cuda.synchronize()
        assert torch.equal(pages, want[0]) and torch.equal(out, want[1])
        assert torch.equal(c.k_means, twin.k_means) and torch.equal(c.k_codes, twin.k_codes)
        assert torch.isfinite(out).all()
