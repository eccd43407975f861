"""Attention over the cache and append under the launch plans that long sequences
and large bounds call for: many splits and their joins, several block lists,
four heads a wave. Rows of no sequence make the bounds large where the work is
small."""

import numpy as np
import pytest

from oracle import kv_cache as R
from tests.gpu_helpers import dev, host, note
from tests.test_gpu_kv_cache import make, tables, widen
from tests.test_gpu_kv_cache_edges import padded

pytestmark = pytest.mark.gpu


def check(i8, rng, cache, table, lens, counts, heads, rows, max_len, splits, rotary=0, **kw):
    """Attention of a batch of `rows` packed rows, bounds of as many new tokens.
    The number of splits is read off the workspace's size: for each row and head
    D + 2 floats a split and a count."""
    kv_heads, dim = cache["k_codes"].shape[1], 16 * cache["k_codes"].shape[3]
    c, b, at, _ = padded(i8, cache, table, lens, counts, rows - sum(counts), rows, max_len)
    need = i8.ops.int8_kv_cache_attention_workspace_bytes(c, b, heads)
    found = (need // 4 // (rows * heads) - 1) // (dim + 2) if need else 1
    assert splits(found), found
    q = np.zeros((rows, heads, dim), np.float16)
    q[at] = rng.normal(0, 1.5, (len(at), heads, dim))
    cos = sin = rot = None
    if rotary:
        cos, sin = tables(rotary, max_len)
        rot = i8.Rotary(dev(cos), dev(sin))
    note("dim=%d rows=%d lens=%s splits=%d" % (dim, rows, lens, found))
    slopes = kw.get("slopes")
    got = host(c.attention(dev(q), b, rot, causal=kw.get("causal", True),
                           window=kw.get("window", 0),
                           alibi_slopes=None if slopes is None else dev(slopes)))
    want, bound = R.attention(cache, q[at], (table, lens, counts), cos, sin, **kw)
    worst = np.max(np.abs(got[at].astype(np.float64) - want) / bound)
    assert worst <= 1.0, worst
    return found


@pytest.mark.parametrize("count", [1, 2, 40])
def test_bound_far_above_the_length(gpu, count):
    """The same work under a close bound and one of 2^20 tokens: other splits."""
    rng = np.random.default_rng(count)
    lens, counts = [2500, 700], [count, 1]
    cache, table = make(rng, lens, 1, 64, 64)
    close = check(gpu, rng, cache, table, lens, counts, 2, count + 1, 2500, lambda s: s > 1)
    cache, table = widen((cache, table), 64)
    check(gpu, rng, cache, table, lens, counts, 2, count + 1, 1 << 20, lambda s: s != close)


@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("kw", [{}, {"window": 5100}, {"rotary": 64}])
def test_few_rows_over_many_splits(gpu, dim, kw):
    """More than 16 splits with tokens in each, among them some without a visible
    one, beside a sequence of one split."""
    rng = np.random.default_rng(dim)
    lens = [6000, 40]
    cache, table = make(rng, lens, 1, dim, 64)
    table[0, 20:40] = -1
    check(gpu, rng, cache, table, lens, [1, 1], 2, 2, 6000, lambda s: s > 16, **kw)


def test_few_rows_over_hundreds_of_splits(gpu):
    rng = np.random.default_rng(2)
    lens = [70000]
    cache, table = make(rng, lens, 1, 64, 128)
    check(gpu, rng, cache, table, lens, [1], 1, 1, 70000, lambda s: s > 256)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kw", [{}, {"window": 7000}, {"alibi": True}])
def test_few_rows_with_several_block_lists(gpu, dim, kw):
    """A bound of 2^23 tokens: chunks of 8 K, of which a wave's list of blocks
    holds 4 K."""
    kw = dict(kw)
    rng = np.random.default_rng(dim + 3)
    lens = [9000, 4200]
    cache, table = make(rng, lens, 1, dim, 64)
    table[0, 70] = -1
    table = np.pad(table, ((0, 0), (0, (1 << 17) - table.shape[1])), constant_values=-1)
    if kw.pop("alibi", False):
        kw["slopes"] = np.array([0.01, 0.001], np.float32)
    check(gpu, rng, cache, table, lens, [1, 1], 2, 2, 1 << 23, lambda s: s > 1000, **kw)


# Head size, rows of the batch, longest sequence, splits: waves of 16 rows, chunks
# below and above a list of 1024 tokens; of 32 rows (16000, 12000 and 4096 rows).
@pytest.mark.parametrize("dim,rows,length,splits", [
    (64, 5600, 2300, 2), (80, 5600, 2300, 2), (96, 5600, 2300, 2), (128, 5600, 2300, 2),
    (64, 8192, 2300, 1), (256, 8192, 2300, 1), (256, 4500, 2300, 2), (256, 2048, 2300, 4),
    (64, 16000, 9000, 2), (80, 12000, 6000, 2), (96, 12000, 6000, 2), (128, 4096, 4200, 4),
    (128, 2000, 1500, 4), (64, 300, 1500, 4)])
@pytest.mark.parametrize("kw", [{}, {"window": 1300}, {"alibi": True, "rotary": 32},
                                {"causal": False}])
def test_many_rows_split_or_in_several_lists(gpu, dim, rows, length, splits, kw):
    kw = dict(kw)
    rng = np.random.default_rng(dim + rows)
    lens, counts = [length, 70, length - 700], [37, 3, 1]
    cache, table = make(rng, lens, 1, dim, 64)
    table[0, 9] = -1
    if kw.pop("alibi", False):
        kw["slopes"] = np.array([0.02, 0.001, 0.1, 0.0], np.float32)
    check(gpu, rng, cache, table, lens, counts, 4, rows, length, lambda s: s == splits, **kw)


@pytest.mark.parametrize("kw", [
    {}, {"causal": False}, {"window": 1}, {"window": 37}, {"rotary": 32}, {"rotary": 64},
    {"alibi": True}, {"alibi": True, "window": 100}])
def test_waves_of_32_rows_of_64_features(gpu, kw):
    """64 features take them under larger bounds than others do."""
    kw = dict(kw)
    rng = np.random.default_rng(64 + len(kw))
    lens, counts = [150, 33, 1, 0, 90, 64, 1200], [150, 1, 1, 0, 0, 17, 70]
    cache, table = widen(make(rng, lens, 4, 64, 64), 64)
    if kw.pop("alibi", False):
        kw["slopes"] = (2.0 ** -np.arange(1, 13)).astype(np.float32)
    check(gpu, rng, cache, table, lens, counts, 12, 300, 1 << 18, lambda s: s < 16, **kw)


@pytest.mark.parametrize("dim,kv_heads", [(64, 5), (80, 6), (96, 7), (128, 5), (256, 6)])
@pytest.mark.parametrize("rotary,interleaved", [(0, False), (32, False), (64, True)])
def test_append_four_heads_a_wave(gpu, dim, kv_heads, rotary, interleaved):
    """A launch of more than 32768 blocks and heads, which do not divide by four;
    bit for bit."""
    rng = np.random.default_rng(dim + kv_heads)
    rows, lens, counts = 7200, [90, 1, 300, 0, 17, 64, 33, 250], [40, 1, 300, 0, 2, 64, 16, 7]
    assert (rows + 30) // 16 * kv_heads * 2 * len(lens) >= 32768
    cache, table = make(rng, lens, kv_heads, dim, 48)
    c, b, at, _ = padded(gpu, cache, table, lens, counts, rows - sum(counts), rows, 300)
    k, v = np.zeros((2, rows, kv_heads, dim), np.float16)
    k[at], v[at] = rng.normal(0, 2, (2, len(at), kv_heads, dim))
    cos = sin = rot = None
    if rotary:
        cos, sin = tables(rotary, 300)
        rot = gpu.Rotary(dev(cos), dev(sin), interleaved)
    note("append, four heads a wave: dim=%d heads=%d" % (dim, kv_heads))
    c.append(dev(k), dev(v), b, rot)
    R.append(cache, k[at], v[at], (table, lens, counts), cos, sin, interleaved)
    for name in ("k_absmax", "v_absmax", "k_codes", "v_codes"):
        assert np.array_equal(host(getattr(c, name)), cache[name],
                              equal_nan=name.endswith("absmax")), name
