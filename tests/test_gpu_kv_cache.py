"""The paged 8-bit key/value cache on the GPU against the numpy reference:
append and read bit for bit, attention within its derived bound."""

import math

import numpy as np
import pytest
import torch

from oracle import kv_cache as R
from tests.gpu_helpers import dev, host, note

pytestmark = pytest.mark.gpu


def make(rng, lens, kv_heads=2, dim=64, page=32, spare=2, poison=True):
    """A cache holding lens[b] tokens of each sequence, and its page table. What
    no token of a sequence stands in holds NaN absmaxes and the largest codes."""
    counts = [-(-int(l) // page) for l in lens]
    pages = sum(counts) + spare
    width = max(counts + [1]) + 1
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    slots = page // 16
    shape = (pages, kv_heads, slots)
    cache = {}
    for w in "kv":
        cache[w + "_codes"] = rng.integers(-127, 128, shape + (dim // 16, 16, 16)).astype(np.int8)
        cache[w + "_absmax"] = np.exp(rng.normal(0, 0.7, shape)).astype(np.float32) * 2
    if poison:
        used = np.zeros(shape, bool)
        for b, l in enumerate(lens):
            for t in range(0, int(l), 16):
                p, s, _ = R.place(cache, table[b], t)
                used[p, :, s] = True
        for w in "kv":
            cache[w + "_absmax"][~used] = np.nan
            cache[w + "_codes"][~used] = 127
    return cache, table


def tables(dim, positions):
    half = dim // 2
    ang = np.arange(positions)[:, None] * (100.0 ** (-np.arange(half) / half))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def on_gpu(i8, cache, table, lens, counts, **kw):
    c = i8.Int8KVCache.from_tensors(*(dev(cache[n]) for n in
                                      ("k_codes", "k_absmax", "v_codes", "v_absmax")))
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    b = i8.KVBatch(dev(table), dev(np.array(lens, np.int32)), dev(cu), total_tokens=int(cu[-1]),
                   max_tokens=max(list(counts) + [0]), **kw)
    return c, b


def check_attention(i8, rng, lens, counts, heads=4, kv_heads=2, dim=64, page=32, rotary=0,
                    interleaved=False, cache=None, q=None, max_len=None, **kw):
    cache, table = cache or make(rng, lens, kv_heads, dim, page)
    total = sum(counts)
    if q is None:
        q = rng.normal(0, 1.5, (total, heads, dim)).astype(np.float16)
    cos = sin = rot = None
    if rotary:
        cos, sin = tables(rotary, max(max(lens), max_len or 0) + 1)
        rot = i8.Rotary(dev(cos), dev(sin), interleaved)
    c, b = on_gpu(i8, cache, table, lens, counts, max_len=max(lens) if max_len is None else max_len)
    slopes = kw.get("slopes")
    got = c.attention(dev(q), b, rot, scale=kw.get("scale"), causal=kw.get("causal", True),
                      window=kw.get("window", 0),
                      alibi_slopes=None if slopes is None else dev(slopes))
    want, bound = R.attention(cache, q, (table, lens, counts), cos, sin, interleaved, **kw)
    got = host(got).astype(np.float64)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / bound) if got.size else 0.0
    assert worst <= 1.0, worst
    return got


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("rotary,interleaved", [(0, False), (1, False), (1, True), (2, False),
                                                (2, True)])
def test_append_and_read_bit_exact(gpu, dim, rotary, interleaved):
    """Prompts, chunks and single tokens that start and end anywhere in a block;
    a fused projection's slices as inputs."""
    rng = np.random.default_rng(dim + rotary)
    lens = [1, 16, 17, 33, 40, 95, 0, 70]
    counts = [1, 16, 1, 33, 7, 60, 0, 3]
    rot_dim = {0: 0, 1: dim, 2: 32}[rotary]
    old = [l - n for l, n in zip(lens, counts)]
    kv_heads, page = 3, 48
    cache, table = make(rng, lens, kv_heads, dim, page)
    # a block that starts with new tokens holds whatever it held before
    for b, (o, l) in enumerate(zip(old, lens)):
        for blk in range(-(-o // 16), -(-l // 16)):
            p, s, _ = R.place(cache, table[b], 16 * blk)
            cache["k_absmax"][p, :, s] = np.nan
            cache["v_absmax"][p, :, s] = np.inf
    total = sum(counts)
    fused = rng.normal(0, 1.5, (total, (2 + 2 * kv_heads) * dim)).astype(np.float16)
    fused[rng.random(fused.shape) < 0.002] *= 20
    k = fused[:, 2 * dim:(2 + kv_heads) * dim].reshape(total, kv_heads, dim)
    v = fused[:, (2 + kv_heads) * dim:].reshape(total, kv_heads, dim)
    cos = sin = rot = None
    if rot_dim:
        cos, sin = tables(rot_dim, 96)
        rot = gpu.Rotary(dev(cos), dev(sin), interleaved)
    c, b = on_gpu(gpu, cache, table, lens, counts, max_len=95)
    f = dev(fused)
    ck = f[:, 2 * dim:(2 + kv_heads) * dim].unflatten(1, (kv_heads, dim))
    cv = f[:, (2 + kv_heads) * dim:].unflatten(1, (kv_heads, dim))
    note("append dim=%d rotary=%d" % (dim, rot_dim))
    for _ in range(2):                                   # repeating changes nothing
        c.append(ck, cv, b, rot)
        torch.cuda.synchronize()
        if _ == 0:
            R.append(cache, k, v, (table, lens, counts), cos, sin, interleaved)
        for name in ("k_absmax", "v_absmax", "k_codes", "v_codes"):
            want = cache[name]
            got = host(getattr(c, name))
            assert np.array_equal(got, want, equal_nan=name.endswith("absmax")), name
    gk, gv = c.read(b)
    wk, wv = R.read(cache, (table, lens, counts))
    assert np.array_equal(host(gk), wk) and np.array_equal(host(gv), wv)


def test_append_token_by_token_equals_reference(gpu):
    """A block filled one token at a time: older codes follow a growing absmax."""
    rng = np.random.default_rng(5)
    cache, table = make(rng, [40], 2, 64, 32)
    cos, sin = tables(64, 40)
    rot = gpu.Rotary(dev(cos), dev(sin))
    start = 8
    lens = torch.tensor([start], dtype=torch.int32, device="cuda")
    c = gpu.Int8KVCache.from_tensors(*(dev(cache[n]) for n in
                                       ("k_codes", "k_absmax", "v_codes", "v_absmax")))
    b = gpu.KVBatch(dev(table), lens, max_len=40)
    x = (rng.normal(0, 1, (2, 32, 2, 64)) * np.linspace(0.5, 3, 32)[:, None, None])
    x = x.astype(np.float16)
    for i in range(32):
        lens.fill_(start + i + 1)
        c.append(dev(x[0, i:i + 1]), dev(x[1, i:i + 1]), b, rot)
        R.append(cache, x[0, i:i + 1], x[1, i:i + 1], (table, [start + i + 1], [1]), cos, sin)
    for name in ("k_absmax", "v_absmax", "k_codes", "v_codes"):
        assert np.array_equal(host(getattr(c, name)), cache[name], equal_nan=True), name


def test_append_head_major_input(gpu):
    """Token and head strides exchanged: [heads, tokens, D] storage."""
    rng = np.random.default_rng(6)
    cache, table = make(rng, [37], 4, 64, 16)
    x = rng.normal(0, 1, (2, 4, 37, 64)).astype(np.float16)
    c, b = on_gpu(gpu, cache, table, [37], [37])
    k, v = dev(x[0]).transpose(0, 1), dev(x[1]).transpose(0, 1)
    c.append(k, v, b)
    R.append(cache, x[0].transpose(1, 0, 2), x[1].transpose(1, 0, 2), (table, [37], [37]))
    for name in ("k_absmax", "v_absmax", "k_codes", "v_codes"):
        assert np.array_equal(host(getattr(c, name)), cache[name], equal_nan=True), name


def test_append_edge_values(gpu):
    """All-zero blocks, tiny absmaxes, and a NaN and an infinity that make their
    block NaN and no other."""
    cache, table = make(np.random.default_rng(7), [64], 1, 64, 64)
    k = np.zeros((64, 1, 64), np.float16)
    k[16:32] = np.float16(6e-8)
    k[33, 0, 5] = np.nan
    k[48:] = 1.0
    k[50, 0, 9] = -np.inf
    v = np.ascontiguousarray(k[::-1])
    c, b = on_gpu(gpu, cache, table, [64], [64])
    c.append(dev(k), dev(v), b)
    gk, gv = (host(t).reshape(4, 16, 64) for t in c.read(b))
    assert not gk[0].any() and (gk[1] == np.float16(6e-8)).all()
    assert np.isnan(gk[2]).all() and np.isnan(gk[3]).all()
    assert np.isnan(gv[0]).all() and np.isnan(gv[1]).all()
    assert (gv[2] == np.float16(6e-8)).all() and not gv[3].any()


def test_absent_pages_and_short_sequences(gpu):
    """Tokens on absent pages are not stored, not seen, and read as 0; so are
    tokens before a sequence's start (more new tokens than its length)."""
    rng = np.random.default_rng(8)
    lens, counts = [70, 5, 48], [70, 9, 20]
    cache, table = make(rng, lens, 2, 64, 16)
    table[0, 1] = -1
    table[0, 3] = 1 << 30
    table[2, 0] = cache["k_absmax"].shape[0]
    before = {n: a.copy() for n, a in cache.items()}
    total = sum(counts)
    k, v = rng.normal(0, 1, (2, total, 2, 64)).astype(np.float16)
    c, b = on_gpu(gpu, cache, table, lens, counts)
    c.append(dev(k), dev(v), b)
    R.append(cache, k, v, (table, lens, counts))
    for name in before:
        assert np.array_equal(host(getattr(c, name)), cache[name], equal_nan=True), name
    wk, wv = R.read(cache, (table, lens, counts))
    gk, gv = c.read(b)
    assert np.array_equal(host(gk), wk) and np.array_equal(host(gv), wv)
    got = check_attention(gpu, rng, lens, counts, page=16, cache=(cache, table))
    assert not got[70:74].any()          # positions below 0 see nothing


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_attention_single_tokens(gpu, dim, group):
    rng = np.random.default_rng(dim * 10 + group)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 128, 200, 0, 331]
    check_attention(gpu, rng, lens, [1] * len(lens), heads=2 * group, dim=dim, page=48,
                    rotary=dim)


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("kw", [
    {}, {"causal": False}, {"window": 1}, {"window": 37}, {"rotary": 32, "interleaved": True},
    {"alibi": True}, {"alibi": True, "window": 100}, {"scale": 0.9}])
def test_attention_chunks(gpu, dim, kw):
    """Prompt chunks of every remainder over cached prefixes, mixed with single
    tokens, an empty sequence and one without new tokens."""
    kw = dict(kw)
    rng = np.random.default_rng(dim + len(kw))
    lens, counts = [150, 33, 1, 0, 90, 64, 200], [150, 1, 1, 0, 0, 17, 70]
    if kw.pop("alibi", False):
        kw["slopes"] = (2.0 ** -np.arange(1, 7)).astype(np.float32)
    check_attention(gpu, rng, lens, counts, heads=6, dim=dim, page=16 * (1 + dim % 3), **kw)


@pytest.mark.parametrize("group", [1, 5, 16, 40])
def test_attention_grouped_heads(gpu, group):
    rng = np.random.default_rng(group)
    check_attention(gpu, rng, [90, 130, 20], [3, 2, 20], heads=group, kv_heads=1, dim=128, page=64,
                    rotary=64)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("count", [16, 17, 32, 33, 48, 49, 128, 129])
def test_attention_row_counts(gpu, dim, count):
    """Rows that just fill a tile, or just do not, of each kernel."""
    rng = np.random.default_rng(dim + count)
    check_attention(gpu, rng, [count + 77, count, 1], [count, count, 1], dim=dim, heads=2)


@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("rotary", [16, 48, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_attention_partial_rotation(gpu, dim, rotary, interleaved):
    rng = np.random.default_rng(dim + rotary)
    check_attention(gpu, rng, [130, 70], [1, 63], dim=dim, heads=2, rotary=rotary,
                    interleaved=interleaved)


@pytest.mark.parametrize("count", [1, 2, 40])
def test_attention_long_axis_split(gpu, count):
    """Few rows over a long cache: several splits of the token axis are joined,
    and a launch bound far above the length changes nothing but their number."""
    rng = np.random.default_rng(count)
    lens, counts = [2500, 700], [count, 1]
    cache = make(rng, lens, 1, 64, 64)
    q = rng.normal(0, 1.5, (count + 1, 2, 64)).astype(np.float16)
    for bound in (2500, 1 << 20):
        check_attention(gpu, rng, lens, counts, heads=2, kv_heads=1, page=64, cache=cache, q=q,
                        rotary=0, max_len=bound)


@pytest.mark.parametrize("count", [1, 30])
def test_attention_value_scales_far_apart(gpu, count):
    """Value absmaxes that differ by 2^60 and more, zeros among them, beside
    large and small logits: each block's weight counts in the row sum whatever
    its values are."""
    rng = np.random.default_rng(11)
    lens = [300, 130]
    cache, table = make(rng, lens, 2, 64, 32)
    a = cache["v_absmax"]
    a *= np.float32(2.0) ** rng.integers(-70, 8, a.shape).astype(np.float32)
    a[rng.random(a.shape) < 0.2] = 0
    check_attention(gpu, rng, lens, [count, count], cache=(cache, table), scale=0.3)


@pytest.mark.parametrize("count", [1, 64])
def test_attention_growing_maximum(gpu, count):
    """Logits that grow along the sequence by far more than fp16 can hold, and
    fall again: rows are rescaled on the way."""
    rng = np.random.default_rng(12)
    cache, table = make(rng, [400], 2, 64, 32)
    q = np.abs(rng.normal(0, 2, (count, 4, 64))).astype(np.float16)
    for t in range(0, 400, 16):
        p, s, _ = R.place(cache, table[0], t)
        cache["k_codes"][p, :, s] = np.abs(cache["k_codes"][p, :, s])
        cache["k_absmax"][p, :, s] = 0.01 * 1.5 ** (t // 16 if t < 250 else 25 - t // 16)
    check_attention(gpu, rng, [400], [count], cache=(cache, table))


# A launch bound of 2^16 or 2^20 tokens calls for the widest tiles, whatever the
# lengths.

def widen(cache_and_table, page):
    cache, table = cache_and_table
    return cache, np.pad(table, ((0, 0), (0, (1 << 20) // page - table.shape[1])),
                         constant_values=-1)


@pytest.mark.parametrize("dim", [64, 80, 96, 128])
@pytest.mark.parametrize("kw", [
    {}, {"causal": False}, {"window": 1}, {"window": 37}, {"rotary": 32, "interleaved": True},
    {"rotary": 64}, {"alibi": True}, {"alibi": True, "window": 100}, {"scale": 0.9}])
def test_wide_tiles_chunks(gpu, dim, kw):
    kw = dict(kw)
    rng = np.random.default_rng(dim + 100 * len(kw))
    lens, counts = [150, 33, 1, 0, 90, 64, 1200], [150, 1, 1, 0, 0, 17, 70]
    if kw.pop("alibi", False):
        kw["slopes"] = (2.0 ** -np.arange(1, 13)).astype(np.float32)
    check_attention(gpu, rng, lens, counts, heads=12, kv_heads=4, dim=dim, page=64, max_len=1 << 16,
                    cache=widen(make(rng, lens, 4, dim, 64), 64), **kw)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("count", [127, 128, 129, 255])
def test_wide_tiles_row_counts(gpu, dim, count):
    rng = np.random.default_rng(dim + count)
    lens = [count + 77, count]
    check_attention(gpu, rng, lens, [count, count], dim=dim, heads=4, kv_heads=4, page=32,
                    max_len=1 << 20, cache=widen(make(rng, lens, 4, dim, 32), 32))


@pytest.mark.parametrize("dim", [64, 128])
def test_wide_tiles_values_and_logits_far_apart(gpu, dim):
    """Values of blocks that differ by 2^60, and logits that grow by far more
    than fp16 can hold."""
    rng = np.random.default_rng(dim + 17)
    lens = [400, 260]
    cache, table = make(rng, lens, 4, dim, 32)
    a = cache["v_absmax"]
    a *= np.float32(2.0) ** rng.integers(-70, 8, a.shape).astype(np.float32)
    a[rng.random(a.shape) < 0.2] = 0
    check_attention(gpu, rng, lens, [200, 260], heads=4, kv_heads=4, dim=dim, scale=0.3,
                    max_len=1 << 20, cache=widen((cache, table), 32))
    cache, table = make(rng, lens, 4, dim, 32)
    q = np.abs(rng.normal(0, 2, (460, 4, dim))).astype(np.float16)
    for b in range(2):
        for t in range(0, lens[b], 16):
            p, s, _ = R.place(cache, table[b], t)
            cache["k_codes"][p, :, s] = np.abs(cache["k_codes"][p, :, s])
            cache["k_absmax"][p, :, s] = 0.01 * 1.5 ** (t // 16 if t < 250 else 25 - t // 16)
    check_attention(gpu, rng, lens, [200, 260], heads=4, kv_heads=4, dim=dim, q=q,
                    max_len=1 << 20, cache=widen((cache, table), 32))


@pytest.mark.parametrize("which", ["k_absmax", "v_absmax"])
def test_wide_tiles_nan_blocks_and_queries(gpu, which):
    rng = np.random.default_rng(18)
    lens, counts = [256], [256]
    cache, table = widen(make(rng, lens, 4, 64, 64), 64)
    q = rng.normal(0, 1, (256, 4, 64)).astype(np.float16)
    q[3] = 0
    want, bound = R.attention(cache, q, (table, lens, counts))
    p, s, _ = R.place(cache, table[0], 160)
    cache[which][p, 1:, s] = np.nan
    q[40, 0, 7] = np.nan
    c, b = on_gpu(gpu, cache, table, lens, counts, max_len=1 << 20)
    got = host(c.attention(dev(q), b)).astype(np.float64)
    bad = np.zeros((256, 4), bool)
    bad[160:, 1:] = bad[40, 0] = True
    assert np.isnan(got[bad]).all()
    assert (np.abs(got - want) <= bound)[~bad].all()


def test_attention_query_layouts(gpu):
    """Slices of a fused projection and head-major storage as queries, an output
    given by the caller, and one-token batches without cu_tokens."""
    rng = np.random.default_rng(13)
    lens = [20, 77, 33]
    cache, table = make(rng, lens, 2, 64, 16)
    x = rng.normal(0, 1, (3, 8, 64)).astype(np.float16)
    want, bound = R.attention(cache, x[:, 2:6], (table, lens, [1, 1, 1]))
    c = gpu.Int8KVCache.from_tensors(*(dev(cache[n]) for n in
                                       ("k_codes", "k_absmax", "v_codes", "v_absmax")))
    b = gpu.KVBatch(dev(table), dev(np.array(lens, np.int32)))
    full = dev(x)
    out = torch.empty((3, 4, 64), dtype=torch.float16, device="cuda")
    major = full[:, 2:6].transpose(0, 1).contiguous().transpose(0, 1)
    for q in (full[:, 2:6], major):
        out.fill_(math.nan)
        assert c.attention(q, b, out=out) is out
        assert (np.abs(host(out) - want) <= bound).all()


def test_attention_zero_and_nan_queries(gpu):
    """A zero query averages the visible values; a NaN or infinite query makes
    its own row NaN and no other."""
    rng = np.random.default_rng(14)
    lens, counts = [100], [100]
    cache, table = make(rng, lens, 1, 64, 32)
    q = rng.normal(0, 1, (100, 2, 64)).astype(np.float16)
    q[3] = 0
    q[40, 0, 7] = np.nan
    q[77, 1, 0] = np.inf
    clean = q.copy()
    clean[40, 0], clean[77, 1] = 0, 0
    want, bound = R.attention(cache, clean, (table, lens, counts))
    c, b = on_gpu(gpu, cache, table, lens, counts)
    got = host(c.attention(dev(q), b)).astype(np.float64)
    bad = np.zeros((100, 2), bool)
    bad[40, 0] = bad[77, 1] = True
    assert np.isnan(got[bad]).all()
    assert (np.abs(got - want) <= bound)[~bad].all()


def test_nan_blocks_reach_only_their_readers(gpu):
    """A block made NaN by its content poisons the rows that see it."""
    rng = np.random.default_rng(15)
    lens, counts = [128], [128]
    for which in ("k_absmax", "v_absmax"):
        cache, table = make(rng, lens, 1, 64, 64)
        q = rng.normal(0, 1, (128, 1, 64)).astype(np.float16)
        want, bound = R.attention(cache, q, (table, lens, counts))
        p, s, _ = R.place(cache, table[0], 80)
        cache[which][p, :, s] = np.nan
        c, b = on_gpu(gpu, cache, table, lens, counts)
        got = host(c.attention(dev(q), b)).astype(np.float64)
        assert (np.abs(got - want) <= bound)[:80].all()
        assert np.isnan(got[80:]).all()


def test_attention_repeats_bit_for_bit(gpu):
    """Same inputs, same bits: eager, on another stream, in a replayed graph
    with other work between the replays, and with a workspace that holds NaN."""
    rng = np.random.default_rng(16)
    lens, counts = [1500, 600, 40], [1, 30, 40]
    cache, table = make(rng, lens, 2, 128, 64)
    c, b = on_gpu(gpu, cache, table, lens, counts, max_len=1500)
    q = dev(rng.normal(0, 1, (71, 8, 128)).astype(np.float16))
    k, v = (dev(rng.normal(0, 1, (71, 2, 128)).astype(np.float16)) for _ in range(2))
    c.append(k, v, b)
    first = c.attention(q, b).clone()
    need = gpu.ops.int8_kv_cache_attention_workspace_bytes(c, b, 8)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.append(k, v, b)
        other = c.attention(q, b)
    s.synchronize()
    assert torch.equal(first, other)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(k, v, b)
        gpu.int8_kv_cache_attention(q, c, b, workspace=ws, out=out)
    for _ in range(3):
        out.fill_(7)
        noise = torch.randn(1 << 20, device="cuda").sum()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out) and bool(torch.isfinite(noise))


def test_nothing_outside_the_outputs_is_written(gpu):
    """Appending leaves every other block as it was; attention and read write
    their rows only."""
    rng = np.random.default_rng(17)
    lens, counts = [90, 31], [20, 1]
    cache, table = make(rng, lens, 2, 80, 32)
    c, b = on_gpu(gpu, cache, table, lens, counts)
    k, v = rng.normal(0, 1, (2, 21, 2, 80)).astype(np.float16)
    R.append(cache, k, v, (table, lens, counts))
    c.append(dev(k), dev(v), b)
    for name in ("k_absmax", "v_absmax", "k_codes", "v_codes"):
        assert np.array_equal(host(getattr(c, name)), cache[name], equal_nan=True), name
    pad = torch.full((21 + 8, 4, 80), 3.0, dtype=torch.float16, device="cuda")
    q = dev(rng.normal(0, 1, (21, 4, 80)).astype(np.float16))
    c.attention(q, b, out=pad[4:25])
    assert (pad[:4] == 3).all() and (pad[25:] == 3).all() and torch.isfinite(pad).all()


def test_empty_calls(gpu):
    """No sequences, no tokens, no pages, no room: nothing faults, queries that
    see nothing get 0."""
    i32 = dict(dtype=torch.int32, device="cuda")
    f16 = dict(dtype=torch.float16, device="cuda")
    c = gpu.Int8KVCache(0, 2, 64)
    b = gpu.KVBatch(torch.zeros((2, 3), **i32), torch.tensor([5, 0], **i32))
    x = torch.ones((2, 2, 64), **f16)
    c.append(x, x, b)
    assert not c.attention(x, b).any()
    k, v = c.read(b)
    assert not k.any() and not v.any()
    b = gpu.KVBatch(torch.zeros((2, 0), **i32), torch.tensor([5, 0], **i32))
    assert not gpu.Int8KVCache(1, 2, 64).attention(x, b).any()
    b = gpu.KVBatch(torch.zeros((0, 1), **i32), torch.zeros((0,), **i32))
    e = torch.empty((0, 2, 64), **f16)
    c = gpu.Int8KVCache(1, 2, 64)
    c.append(e, e, b)
    assert c.attention(e, b).shape == (0, 2, 64) and c.read(b)[0].shape == (0, 2, 64)


def test_offsets_beyond_32_bits(gpu):
    """Pages more than 4 GiB into the cache, and tokens more than 4 GiB apart:
    the results of a small cache and of packed tensors, bit for bit."""
    rng = np.random.default_rng(21)
    pages, heads, dim, page = 70000, 8, 128, 64          # 4.6 GB of codes each
    lens, counts = [100, 37], [60, 37]
    far = gpu.Int8KVCache(pages, heads, dim, page)
    near = gpu.Int8KVCache(4, heads, dim, page)
    cu = dev(np.array([0, 60, 97], np.int32))
    b_near = gpu.KVBatch(dev(np.array([[0, 1], [2, 3]], np.int32)), dev(np.array(lens, np.int32)),
                         cu, total_tokens=97, max_tokens=60)
    b_far = gpu.KVBatch(dev(np.array([[pages - 1, 3], [pages - 2, 0]], np.int32)),
                        dev(np.array(lens, np.int32)), cu, total_tokens=97, max_tokens=60)
    x = [dev(rng.normal(0, 1, (97, heads, dim)).astype(np.float16)) for _ in range(3)]
    step = (1 << 31) // 64 + 8                           # elements: 97 of them are 6.5 GB
    room = torch.empty((96 * step + heads * dim,), dtype=torch.float16, device="cuda")
    got = []
    for cache, batch, spread in ((near, b_near, False), (far, b_far, True)):
        cache.k_absmax.zero_()
        cache.v_absmax.zero_()
        cache.k_codes[batch.page_table.long().flatten()] = 0
        cache.v_codes[batch.page_table.long().flatten()] = 0
        q, k, v = x
        if spread:
            view = room.as_strided((97, heads, dim), (step, dim, 1))
        cache.append(view.copy_(k) if spread else k, v, batch)
        cache.append(k, view.copy_(v) if spread else v, batch)
        got.append((*cache.read(batch), cache.attention(view.copy_(q) if spread else q, batch)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
