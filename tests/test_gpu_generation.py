"""Beam searches over the cache, and long sequences with chosen pages: selection, page
tables, copies, append, choice and attention together, through Int8CachedAttention."""

import numpy as np
import pytest
import torch

from oracle import beam as RB
from oracle import kv_sparse as RS
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


class Model:
    """An embedding, two attention layers and a vocabulary, seeded."""

    def __init__(self, i8, rng, hidden=256, heads=4, kv_heads=2, dim=64, vocab=301):
        self.embed = dev(rng.normal(0, 1, (vocab, hidden)).astype(np.float16))
        self.head = i8.Int8Linear(hidden, vocab)
        self.head.quantize_(dev(rng.normal(0, 0.2, (vocab, hidden)).astype(np.float16)))
        self.layers = []
        for _ in range(2):
            layer = i8.Int8CachedAttention(hidden, heads, kv_heads, dim)
            layer.quantize_(*(dev(rng.normal(0, 1 / 16, s).astype(np.float16)) for s in (
                (layer.qkv.out_features, hidden), (hidden, heads * dim))))
            self.layers.append(layer)
        ang = np.arange(512)[:, None] * (100.0 ** (-np.arange(dim // 2) / (dim // 2)))
        self.rot = i8.Rotary(dev(np.cos(ang).astype(np.float32)), dev(np.sin(ang).astype(np.float32)))

    def __call__(self, tokens, caches, batch, choice=None):
        x = self.embed[tokens.clamp(min=0).long()]
        for layer, cache in zip(self.layers, caches):
            x = x + layer(x, cache, batch, self.rot, choice=choice)
        return x


def prompts(i8, model, rng, pool, caches, lens, limit):
    """The prompts' pages and the logits of their last tokens."""
    rows = len(lens)
    table, zero = pool.empty_table(rows, limit)
    none = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    table, seq_lens, _ = pool.step(table, zero, none, new_tokens=dev(np.array(lens, np.int32)))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    batch = i8.KVBatch(table, seq_lens, dev(cu), total_tokens=int(cu[-1]), max_tokens=max(lens),
                       max_len=limit)
    words = dev(rng.integers(0, model.embed.shape[0], int(cu[-1])).astype(np.int32))
    x = model(words, caches, batch)[dev(cu[1:].astype(np.int64)) - 1]
    return table, seq_lens, model.head(x).view(rows, 1, -1)


def test_beam_search_equals_beams_on_their_own(gpu):
    """Beams that share pages give what beams with caches of their own give: the
    logits bit for bit, the choices by the reference."""
    rng = np.random.default_rng(1)
    model, beams, lens, limit, page = Model(gpu, rng), 4, [33, 7], 80, 16
    pool = gpu.KVPages(60, page)
    caches = [gpu.Int8KVCache(60, 2, 64, page) for _ in range(2)]
    table, seq_lens, logits = prompts(gpu, model, rng, pool, caches, lens, limit)
    width = table.shape[1]
    # a cache of its own for each beam: the prompt's pages copied to rows of their own
    alone = [gpu.Int8KVCache(2 * beams * width, 2, 64, page) for _ in range(2)]
    own_table = torch.arange(2 * beams * width, dtype=torch.int32, device="cuda").view(2 * beams, width)
    for a, c in zip(alone, caches):
        for name in ("k_codes", "k_absmax", "v_codes", "v_absmax"):
            src = getattr(c, name)[table.clamp(min=0).long()]           # [2, width, ...]
            getattr(a, name).copy_(src.repeat_interleave(beams, 0).flatten(0, 1))
    search = gpu.BeamSearch(pool, caches, table, seq_lens, beams, eos=2, max_len=limit)
    own_lens = seq_lens.repeat_interleave(beams)
    scores, live = np.zeros((2, 1), np.float32), np.ones((2, 1), np.int32)
    history = []
    for step in range(20):
        want = RB.select(host(logits), scores, live, 2, beams)
        assert want[-1].min() > 2 ** -17
        tokens = search.step(logits)
        assert np.array_equal(host(tokens), want[1]) and np.array_equal(host(search.live), want[3])
        scores, live = host(search.scores), host(search.live)
        assert int(search.wanting) == 0
        history.append((want[1], want[2]))
        # the other caches: each beam's pages become its parent's
        parent = dev(want[2].reshape(-1).astype(np.int64))
        if step:
            for a in alone:
                for name in ("k_codes", "k_absmax", "v_codes", "v_absmax"):
                    x = getattr(a, name).view((2 * beams, width) + getattr(a, name).shape[1:])
                    x.copy_(x[parent].clone())
            own_lens = own_lens[parent]
        own_lens = own_lens + search.live.view(-1)
        own = gpu.KVBatch(own_table, own_lens * search.live.view(-1), max_len=limit)
        assert torch.equal(search.seq_lens, own_lens)
        flat = tokens.view(-1)
        x = model(flat, caches, search.batch)
        y = model(flat, alone, own)
        assert torch.equal(x, y), step
        logits = model.head(x).view(2, beams, -1).clone()
        if step % 5 == 3:
            logits[:, 1, 2] = logits[:, 1].max() + 4     # a beam likely to end
    assert (live == 0).any() and (live == 1).any()
    words, final = search.result()
    words = host(words)
    for s in range(2):
        for i in range(beams):
            at, line = s * beams + i, []
            for tokens, parents in reversed(history):
                line.append(tokens.reshape(-1)[at])
                at = parents.reshape(-1)[at]
            assert words[s, i].tolist() == line[::-1]
    assert np.array_equal(host(final), scores)


def test_search_without_candidates_and_pages(gpu):
    """A search whose logits leave fewer candidates than beams; a pool too small."""
    rng = np.random.default_rng(2)
    model, page = Model(gpu, rng, vocab=5), 16
    pool = gpu.KVPages(3, page)
    caches = [gpu.Int8KVCache(3, 2, 64, page) for _ in range(2)]
    table, seq_lens, logits = prompts(gpu, model, rng, pool, caches, [16], 64)
    logits = logits.clone()
    logits[:, :, 3:] = float("-inf")
    search = gpu.BeamSearch(pool, caches, table, seq_lens, 4, max_len=64)
    tokens = search.step(logits)
    assert host(tokens)[0, 3] == -1 and host(search.live).tolist() == [[1, 1, 1, 0]]
    assert host(search.seq_lens).tolist() == [17, 17, 17, 0]
    # 3 pages: the prompt's and two new ones; the third beam's token is absent
    assert int(search.wanting) == 1 and host(search.page_table)[2, 1] == -1
    x = model(tokens.view(-1), caches, search.batch)
    assert torch.isfinite(x).all()
    with pytest.raises(ValueError):
        gpu.BeamSearch(pool, [gpu.Int8KVCache(2, 2, 64, page)], table, seq_lens, 4)
    with pytest.raises(ValueError):
        gpu.BeamSearch(pool, caches, table, seq_lens, 65)
    with pytest.raises(ValueError):
        gpu.BeamSearch(pool, caches, table, seq_lens, 4).result()


def test_layer_with_chosen_pages(gpu):
    """A prompt in chunks and tokens after it, each attending to chosen pages; the
    means follow the appends, the layer's parts the references."""
    rng = np.random.default_rng(3)
    model, page, limit = Model(gpu, rng), 16, 256
    layer = model.layers[0]
    seen = {}
    layer.qkv.register_forward_hook(lambda m, x, y: seen.update(y=y))
    layer.out.register_forward_hook(lambda m, x, y: seen.update(a=x[0]))
    cache = gpu.Int8KVCache(20, 2, 64, page, page_means=True)
    for x in (cache.k_codes, cache.v_codes, cache.k_absmax, cache.v_absmax):
        x.zero_()
    table = dev(rng.permutation(20)[:16].reshape(1, 16).astype(np.int32))
    choice = gpu.PageChoice(4, first=1, recent=2)
    length = 0
    for n in (100, 37, 1, 1):
        length += n
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        batch = gpu.KVBatch(table, lens, cu, total_tokens=n, max_len=limit)
        layer(dev(rng.normal(0, 1, (n, 256)).astype(np.float16)), cache, batch, model.rot, choice=choice)
        ref = {k: host(getattr(cache, k)) for k in ("k_codes", "k_absmax", "v_codes", "v_absmax")}
        means = np.zeros(cache.k_means.shape, np.float16)
        b_ref = (host(table), [length], [n])
        RS.page_means(ref, means, (host(table), [length], [length]))
        held = host(table)[0, :-(-length // page)]
        assert np.array_equal(host(cache.k_means)[held], means[held])
        q = host(seen["y"]).reshape(n, -1, 64)[:, :4]
        cos, sin = host(model.rot.cos), host(model.rot.sin)
        pages, gap = RS.select_pages(ref, means, q, b_ref, 4, 1, 2, cos, sin)
        assert gap > 1e-9
        want, bound = RS.attention_pages(ref, q, b_ref, pages, cos, sin)
        got = host(seen["a"]).reshape(want.shape).astype(np.float64)
        assert (np.abs(got - want) <= bound).all()
    with pytest.raises(ValueError):
        layer(torch.zeros((1, 256), dtype=torch.float16, device="cuda"), cache, batch, model.rot, window=5,
              choice=choice)
    with pytest.raises(ValueError, match="mean keys"):
        plain = gpu.Int8KVCache(20, 2, 64, page)
        batch = gpu.KVBatch(table, lens, max_len=limit)
        layer(torch.zeros((1, 256), dtype=torch.float16, device="cuda"), plain, batch, model.rot,
              choice=choice)


def test_forked_cache_with_means(gpu):
    """Copies take the mean keys with them; after compaction the choice names the
    same pages of a sequence and the attention is the same."""
    rng = np.random.default_rng(4)
    page, heads = 32, 2
    pool = gpu.KVPages(40, page)
    cache = gpu.Int8KVCache(40, heads, 64, page, page_means=True)
    table, zero = pool.empty_table(3, 400)
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    lens = [300, 90, 170]
    table, seq_lens, _ = pool.step(table, zero, none, new_tokens=dev(np.array(lens, np.int32)))
    kv = dev(rng.normal(0, 1, (2, sum(lens), heads, 64)).astype(np.float16))
    cu = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    cache.append(kv[0], kv[1], gpu.KVBatch(table, seq_lens, cu, total_tokens=sum(lens), max_tokens=300,
                                           max_len=400))
    # the second ends, the first goes on twice
    table, seq_lens, copies = pool.step(table, seq_lens, torch.tensor([0, 0, 2], dtype=torch.int32,
                                                                      device="cuda"))
    cache.copy_pages(copies)
    batch = gpu.KVBatch(table, seq_lens, max_len=400)
    cache.append(*dev(rng.normal(0, 1, (2, 3, heads, 64)).astype(np.float16)), batch)
    q = dev(rng.normal(0, 1, (3, 4, 64)).astype(np.float16))

    def look():
        pages = cache.select_pages(q, batch, 5, recent=2)
        return pages, cache.attention_pages(q, pages, batch), cache.attention(q, batch)
    before = look()
    table, copies = pool.compact(table, seq_lens)
    cache.copy_pages(copies)
    used = int(copies.counts[1])
    assert used == 10 + 1 + 6 and int(host(table).max()) == used - 1
    for x in (cache.k_absmax, cache.v_absmax, cache.k_means):
        x[used:] = float("nan")
    batch = gpu.KVBatch(table, seq_lens, max_len=400)
    for a, b in zip(before, look()):
        assert torch.equal(a, b)
