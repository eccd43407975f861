"""The paged 8-bit key/value cache where sizes and contents meet limits."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as R
from tests.gpu_helpers import dev, host, note
from tests.test_gpu_cached_attention import build, empty_cache
from tests.test_gpu_kv_cache import check_attention, make, on_gpu, tables, widen

pytestmark = pytest.mark.gpu


# ------------------------------------------- packed rows without a sequence

def padded(i8, cache, table, lens, counts, extra, max_tokens, max_len):
    """A batch with `extra` rows past the last sequence's, each sequence's new
    tokens cut to max_tokens. Also the rows that belong to a sequence, and how
    many of each sequence's do."""
    c = i8.Int8KVCache.from_tensors(*(dev(cache[n]) for n in
                                      ("k_codes", "k_absmax", "v_codes", "v_absmax")))
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    b = i8.KVBatch(dev(table), dev(np.array(lens, np.int32)), dev(cu),
                   total_tokens=int(cu[-1]) + extra, max_tokens=max_tokens, max_len=max_len)
    kept = [min(n, max_tokens) for n in counts]
    rows = np.concatenate([np.arange(s, s + n) for s, n in zip(cu, kept)]).astype(int)
    return c, b, rows, kept


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("counts,max_tokens", [
    ([1, 1, 1], 1), ([3, 0, 1], 3), ([70, 1, 33], 70), ([70, 1, 33], 40), ([9, 1, 2], 4),
    ([5, 2, 90], 64)])
@pytest.mark.parametrize("splits", [False, True])
def test_rows_of_no_sequence_are_zero(gpu, dim, counts, max_tokens, splits):
    """Rows past the last sequence's and tokens beyond max_tokens give 0 from
    attention and read, whatever the outputs and the workspace held."""
    rng = np.random.default_rng(dim + sum(counts) + max_tokens)
    lens = [200, 1, 640]
    heads, kv_heads = 4, 2
    cache, table = make(rng, lens, kv_heads, dim, 64)
    if splits:      # a bound far above the lengths: many splits, which only few sequences fill
        table = np.pad(table, ((0, 0), (0, 256 - table.shape[1])), constant_values=-1)
    c, b, rows, kept = padded(gpu, cache, table, lens, counts, 21, max_tokens,
                              64 * table.shape[1])
    total = b.total_tokens
    q = rng.normal(0, 1, (total, heads, dim)).astype(np.float16)
    want, bound = R.attention(cache, q[rows], (table, lens, kept))
    owned = np.zeros(total, bool)
    owned[rows] = True
    wk, wv = R.read(cache, (table, lens, kept))
    need = gpu.ops.int8_kv_cache_attention_workspace_bytes(c, b, heads)
    lib = gpu.load_library()
    note("rows of no sequence: dim=%d counts=%s max_tokens=%d" % (dim, counts, max_tokens))
    for poison in (1, 65):       # of the workspace: counts far above the splits, floats 2e-38 and 12
        ws = torch.full((max(need, 1),), poison, dtype=torch.uint8, device="cuda")
        out = torch.full((total, heads, dim), 1000.0, dtype=torch.float16, device="cuda")
        got = host(gpu.ops.int8_kv_cache_attention(dev(q), c, b, workspace=ws, out=out))
        assert (np.abs(got[owned].astype(np.float64) - want) <= bound).all()
        assert not got[~owned].any()
    k, v = torch.full((2, total, kv_heads, dim), 1000.0, dtype=torch.float16, device="cuda")
    assert lib.int8_kv_cache_read(c.ref, b.ref, k.data_ptr(), v.data_ptr(),
                                  torch.cuda.current_stream().cuda_stream) == 0
    assert np.array_equal(host(k)[rows], wk) and np.array_equal(host(v)[rows], wv)
    assert not host(k)[~owned].any() and not host(v)[~owned].any()


def test_layer_ignores_rows_of_no_sequence(gpu):
    """The output projection picks its outlier columns over all rows: padded ones
    give it zeros, so the rows of sequences do not depend on what memory held."""
    rng = np.random.default_rng(3)
    layer, seen, _ = build(gpu, rng, 256, 4, 2, 64)
    table = np.arange(12, dtype=np.int32).reshape(2, 6)
    x = np.zeros((64, 256), np.float16)
    x[:31] = rng.normal(0, 1, (31, 256))
    outs = []
    for poison in (0.0, 1000.0):
        cache, _ = empty_cache(gpu, 12, 2, 64, 32)
        b = gpu.KVBatch(dev(table), dev(np.array([30, 1], np.int32)),
                        dev(np.array([0, 30, 31], np.int32)), total_tokens=64, max_tokens=40)
        # every block that the step may be given holds the poison
        held = [torch.full((n,), poison, dtype=torch.float16, device="cuda")
                for n in (64 * 256, 64 * 512, 1 << 18, 1 << 20) for _ in range(6)]
        del held
        outs.append(host(layer(dev(x), cache, b))[:31])
        assert not host(seen["a"])[31:].any()
    assert np.array_equal(*outs)


# ---------------------------------------------------------- infinite queries

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("count,heads", [(1, 2), (60, 2), (200, 4)])
def test_infinite_query_is_nan_whatever_the_keys(gpu, interleaved, value, count, heads):
    """A rotated query with an infinity, over keys of one sign: its row is NaN
    where it sees a token and 0 where it sees none; no other row changes."""
    rng = np.random.default_rng(31)
    lens, dim = [count + 3], 64
    for sign in (1, -1):
        cache, table = make(rng, lens, 1, dim, 64)
        cache["k_codes"] = (sign * np.maximum(np.abs(cache["k_codes"]), 1)).astype(np.int8)
        q = np.abs(rng.normal(0, 1, (count, heads, dim))).astype(np.float16)
        cos, sin = tables(dim, lens[0] + 1)
        rot = gpu.Rotary(dev(cos), dev(sin), interleaved)
        want, bound = R.attention(cache, q, (table, lens, [count]), cos, sin, interleaved)
        bad = np.zeros((count, heads), bool)
        for i in {0, count // 2, count - 1}:
            bad[i, i % heads] = True
            q[i, i % heads, 6] = value
        c, b = on_gpu(gpu, cache, table, lens, [count], max_len=lens[0])
        got = host(c.attention(dev(q), b, rot)).astype(np.float64)
        assert np.isnan(got[bad]).all()
        assert (np.abs(got - want) <= bound)[~bad].all()
        absent = np.full_like(table, -1)
        c, b = on_gpu(gpu, cache, absent, lens, [count], max_len=lens[0])
        assert not host(c.attention(dev(q), b, rot)).any()


# ------------------------------------------------------------ recorded steps

def test_recorded_step_after_larger_calls(gpu):
    """A recorded step, then larger eager calls on the stream it was recorded on,
    which replace the stream's shared workspace: the replays give what they gave,
    and write to nothing else."""
    rng = np.random.default_rng(51)
    layer, _, _ = build(gpu, rng, 256, 4, 2, 64)
    cache, _ = empty_cache(gpu, 160, 2, 64, 64)
    table = dev(np.arange(160, dtype=np.int32).reshape(2, 80))
    prompt = gpu.KVBatch(table, dev(np.array([4000, 1500], np.int32)),
                         dev(np.array([0, 4000, 5500], np.int32)), total_tokens=5500,
                         max_tokens=4000)
    tokens = gpu.KVBatch(table, dev(np.array([4001, 1501], np.int32)))
    many = dev(rng.normal(0, 1, (5500, 256)).astype(np.float16))
    x = dev(rng.normal(0, 1, (2, 256)).astype(np.float16))
    layer(many, cache, prompt)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = layer(x, cache, tokens).clone()
        layer(x, cache, tokens)
    side.synchronize()
    assert gpu.ops.int8_kv_cache_attention_workspace_bytes(cache, tokens, 4) > 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = layer(x, cache, tokens)
    for _ in range(3):
        with torch.cuda.stream(side):
            layer(many, cache, prompt)
            layer(x, cache, tokens)
            # whatever the stream's allocator has free now belongs to these
            others = [torch.full((n,), 77, dtype=torch.uint8, device="cuda")
                      for n in (1 << 10, 1 << 14, 1 << 17, 1 << 19, 1 << 20, 1 << 22, 1 << 24)
                      for _ in range(4)]
            y.fill_(5)
            g.replay()
        side.synchronize()
        assert torch.equal(y, want)
        assert all(bool((t == 77).all()) for t in others)
        del others


# ------------------------------------------------------------- empty batches

@pytest.mark.parametrize("max_tokens", [0, 5])
@pytest.mark.parametrize("seqs", [0, 2])
def test_padding_alone(gpu, seqs, max_tokens):
    """No sequences, or none with new tokens: append does nothing, every row of
    attention and read is 0."""
    i32 = dict(dtype=torch.int32, device="cuda")
    c = gpu.Int8KVCache(2, 2, 64)
    for t in (c.k_codes, c.v_codes, c.k_absmax, c.v_absmax):
        t.fill_(3)
    b = gpu.KVBatch(torch.zeros((seqs, 1), **i32), torch.full((seqs,), 9, **i32),
                    torch.zeros((seqs + 1,), **i32), total_tokens=5, max_tokens=max_tokens)
    x = torch.ones((5, 2, 64), dtype=torch.float16, device="cuda")
    c.append(x, x, b)
    assert all((t == 3).all() for t in (c.k_codes, c.v_codes, c.k_absmax, c.v_absmax))
    out = torch.full((5, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    assert not c.attention(x.repeat(1, 2, 1), b, out=out).any()
    held = [torch.full_like(x, 7.0) for _ in range(4)]     # what read is given next holds 7
    del held
    k, v = c.read(b)
    assert k.shape == x.shape and not k.any() and not v.any()


# ------------------------------------------------------------ many sequences

def test_many_sequences_with_a_wide_bound(gpu):
    """60000 single tokens whose launch bound is the packed rows' total: the work
    is small, and so is the launch. Against the same sequences a few at a time."""
    rng = np.random.default_rng(41)
    seqs, total, heads, dim, page = 60000, 80000, 64, 64, 16
    cache, _ = make(rng, [16 * 40], 1, dim, page, spare=0)
    table = rng.integers(0, 40, (seqs, 1)).astype(np.int32)       # shared pages
    lens = rng.integers(1, 17, seqs).astype(np.int32)
    c = gpu.Int8KVCache.from_tensors(*(dev(cache[n]) for n in
                                       ("k_codes", "k_absmax", "v_codes", "v_absmax")))
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    b = gpu.KVBatch(dev(table), dev(lens), cu, total_tokens=total)
    q = torch.randn((total, heads, dim), dtype=torch.float16, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(1))
    note("60000 sequences")
    got = c.attention(q, b)
    assert not got[seqs:].any()
    some = np.unique(np.concatenate([[0, 1, 63, 64, 65, 4095, 4096, seqs - 2, seqs - 1],
                                     rng.integers(0, seqs, 40)]))
    at = torch.from_numpy(some).cuda()
    want, bound = R.attention(cache, host(q[at]), (table[some], lens[some], [1] * len(some)))
    assert (np.abs(host(got[at]).astype(np.float64) - want) <= bound).all()


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("seqs", [65, 130, 300])
@pytest.mark.parametrize("kw", [{}, {"window": 50}, {"wide": True}])
def test_more_sequences_than_a_wave_has_lanes(gpu, dim, seqs, kw):
    """Single tokens, chunks and sequences without new tokens, more than 64 of
    them, over prefixes of several splits."""
    kw = dict(kw)
    rng = np.random.default_rng(seqs + dim)
    counts = rng.choice([0, 1, 1, 1, 2], seqs)
    counts[rng.choice(seqs, 3, replace=False)] = [40, 129, 90]
    counts[-1] = 65
    lens = counts + rng.integers(0, 30, seqs)
    lens[[0, seqs // 2, seqs - 1]] += 1100
    counts, lens = counts.tolist(), lens.tolist()
    cache = make(rng, lens, 2, dim, 32)
    if kw.pop("wide", False):
        cache, kw["max_len"] = widen(cache, 32), 1 << 20
    check_attention(gpu, rng, lens, counts, heads=4, dim=dim, page=32, cache=cache, **kw)


@pytest.mark.parametrize("cut", [0, 7])
def test_many_sequences_of_one_token_or_cut(gpu, cut):
    """65 and more sequences without cu_tokens, and with new tokens beyond
    max_tokens, of 64 query heads on one."""
    rng = np.random.default_rng(61 + cut)
    seqs, heads, dim = 90, 64, 64
    lens = rng.integers(1, 200, seqs).tolist()
    cache, table = make(rng, lens, 1, dim, 16)
    if not cut:
        q = rng.normal(0, 1, (seqs, heads, dim)).astype(np.float16)
        c, _, _, _ = padded(gpu, cache, table, lens, [1] * seqs, 0, 1, 200)
        b = gpu.KVBatch(dev(table), dev(np.array(lens, np.int32)), max_len=200)
        rows, kept = np.arange(seqs), [1] * seqs
    else:
        counts = rng.integers(0, 2 * cut, seqs).tolist()
        c, b, rows, kept = padded(gpu, cache, table, lens, counts, 3, cut, 200)
        q = rng.normal(0, 1, (b.total_tokens, heads, dim)).astype(np.float16)
    want, bound = R.attention(cache, q[rows], (table, lens, kept))
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    got = host(c.attention(dev(q), b, out=out)).astype(np.float64)
    assert (np.abs(got[rows] - want) <= bound).all()
    assert not np.delete(got, rows, axis=0).any()


# ---------------------------------------- weights far below a row's largest

@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_small_weights_beside_a_large_one(gpu, dim):
    """131000 tokens of weight 2^-25.5 beside one of weight 1, every value the
    same: the result is that value. Rounded: the output (2^-11 relative) and the
    weights (2^-11); a chain of binary32 sums over the tokens, 32 an addition,
    above and below the line (2^-24 each). Together the small weights are 0.0027
    of the sum, so they have to count on both sides."""
    length, count = 131000, 64
    page, pages = 64, -(-length // 64)
    slots, tiles = page // 16, dim // 16
    cache = {"k_codes": np.zeros((pages, 1, slots, tiles, 16, 16), np.int8),
             "k_absmax": np.ones((pages, 1, slots), np.float32),
             "v_codes": np.full((pages, 1, slots, tiles, 16, 16), 127, np.int8),
             "v_absmax": np.ones((pages, 1, slots), np.float32)}
    cache["k_codes"][0, 0, 0, 0, 0, 0] = 127                 # token 0, feature 0
    table = np.full((1, 1 << 20), -1, np.int32)              # a bound of 2^26: few splits
    table[0, :pages] = np.arange(pages)
    q = np.zeros((count, 4, dim), np.float16)
    q[:, :, 0] = 1
    c, b = on_gpu(gpu, cache, table, [length], [count])
    got = host(c.attention(dev(q), b, scale=25.5 * float(np.log(2)))).astype(np.float64)
    tol = 2.0 ** -11 + 2.0 ** -11 + 2 * length / 32 * 2.0 ** -24
    assert np.abs(got - 1).max() <= tol, np.abs(got - 1).max()


@pytest.mark.parametrize("count", [1, 60])
def test_empty_rotation_tables_are_not_read(gpu, count):
    """Tables of no positions serve a batch without room for tokens: their
    addresses are never followed."""
    i32 = dict(dtype=torch.int32, device="cuda")
    c = gpu.Int8KVCache(1, 2, 64)
    b = gpu.KVBatch(torch.zeros((1, 1), **i32), torch.full((1,), 5, **i32),
                    torch.tensor([0, count], **i32), total_tokens=count, max_len=0)
    rot = gpu.Rotary(torch.zeros((0, 32), device="cuda"), torch.zeros((0, 32), device="cuda"))
    rot._struct.cos = rot._struct.sin = 0x10000
    x = torch.ones((count, 4, 64), dtype=torch.float16, device="cuda")
    out = torch.full_like(x, 7.0)
    assert not c.attention(x, b, rot, out=out).any()
    c.append(x[:, :2], x[:, 2:], b, rot)
