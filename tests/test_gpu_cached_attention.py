"""Int8CachedAttention: the projections, the cache and the attention together,
stage by stage against the oracles."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as R
from oracle import llm_int8 as O
from tests.gpu_helpers import Y_TOL, dev, host, y_err

pytestmark = pytest.mark.gpu


def batches(i8, table, lens, counts, max_len):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ref = (table, lens, counts)
    if all(c == 1 for c in counts):
        return ref, i8.KVBatch(dev(table), dev(np.array(lens, np.int32)), max_len=max_len)
    return ref, i8.KVBatch(dev(table), dev(np.array(lens, np.int32)), dev(cu),
                           total_tokens=int(cu[-1]), max_tokens=max(counts), max_len=max_len)


def build(i8, rng, hidden, heads, kv_heads, dim):
    layer = i8.Int8CachedAttention(hidden, heads, kv_heads, dim, bias=True)
    w_qkv = rng.normal(0, 1 / np.sqrt(hidden), (layer.qkv.out_features, hidden)).astype(np.float16)
    w_out = rng.normal(0, 1 / np.sqrt(heads * dim), (hidden, heads * dim)).astype(np.float16)
    b = [rng.normal(0, 0.1, n).astype(np.float16) for n in (layer.qkv.out_features, hidden)]
    layer.quantize_(dev(w_qkv), dev(w_out), dev(b[0]), dev(b[1]))
    seen = {}
    layer.qkv.register_forward_hook(lambda m, x, y: seen.update(x=x[0], y=y))
    layer.out.register_forward_hook(lambda m, x, y: seen.update(a=x[0], z=y))
    refs = [O.quantize_weight_rows(w) + (bb,) for w, bb in zip((w_qkv, w_out), b)]
    return layer, seen, refs


def empty_cache(i8, pages, kv_heads, dim, page):
    cache = i8.Int8KVCache(pages, kv_heads, dim, page)
    ref = {"k_codes": np.zeros(cache.k_codes.shape, np.int8),
           "k_absmax": np.zeros(cache.k_absmax.shape, np.float32),
           "v_codes": np.zeros(cache.v_codes.shape, np.int8),
           "v_absmax": np.zeros(cache.v_absmax.shape, np.float32)}
    return cache, ref


@pytest.mark.parametrize("hidden,heads,kv_heads,dim,rotary,alibi,window", [
    (256, 4, 4, 64, 64, False, 0), (320, 8, 2, 80, 32, False, 40), (512, 4, 1, 128, 0, True, 0)])
def test_prompts_then_tokens(gpu, hidden, heads, kv_heads, dim, rotary, alibi, window):
    """Ragged prompts, the rest of one of them beside single tokens of the
    others, then single tokens of all: the stored cache bit for bit, every
    stage's output within its own bound."""
    rng = np.random.default_rng(hidden)
    layer, seen, refs = build(gpu, rng, hidden, heads, kv_heads, dim)
    page, limit = 32, 224
    cache, ref = empty_cache(gpu, 22, kv_heads, dim, page)
    table = rng.permutation(22)[:21].reshape(3, 7).astype(np.int32)
    rot = cos = sin = slopes = None
    if rotary:
        ang = np.arange(limit)[:, None] * (100.0 ** (-np.arange(rotary // 2) / (rotary // 2)))
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        rot = gpu.Rotary(dev(cos), dev(sin))
    if alibi:
        slopes = (2.0 ** -np.arange(1, heads + 1)).astype(np.float32)
    lens = [0, 0, 0]
    for counts in ([70, 1, 129], [33, 1, 1], [1, 1, 1], [1, 1, 1]):
        lens = [l + c for l, c in zip(lens, counts)]
        b_ref, b = batches(gpu, table, lens, counts, limit)
        x = rng.normal(0, 1, (sum(counts), hidden)).astype(np.float16)
        x[:, 5] *= 12      # an outlier feature
        z = host(layer(dev(x), cache, b, rot, window=window,
                       alibi_slopes=None if slopes is None else dev(slopes)))
        y, a = host(seen["y"]), host(seen["a"])
        (wq, sw, bias), (wq2, sw2, bias2) = refs
        assert y_err(y, O.linear_int8_mixed(x, wq, sw, bias=bias)["Y"]) <= Y_TOL
        q, k, v = np.split(y.reshape(len(y), -1, dim), [heads, heads + kv_heads], axis=1)
        R.append(ref, k, v, b_ref, cos, sin)
        gk, gv = cache.read(b)
        wk, wv = R.read(ref, b_ref)
        assert np.array_equal(host(gk), wk) and np.array_equal(host(gv), wv)
        want, bound = R.attention(ref, q, b_ref, cos, sin, window=window, slopes=slopes)
        assert (np.abs(a.reshape(want.shape).astype(np.float64) - want) <= bound).all()
        assert y_err(z, O.linear_int8_mixed(a, wq2, sw2, bias=bias2)["Y"]) <= Y_TOL


def test_empty_step(gpu):
    rng = np.random.default_rng(1)
    layer, _, _ = build(gpu, rng, 256, 4, 4, 64)
    cache, _ = empty_cache(gpu, 2, 4, 64, 32)
    _, b = batches(gpu, np.zeros((2, 1), np.int32), [3, 0], [0, 0], 32)
    assert layer(torch.empty((0, 256), dtype=torch.float16, device="cuda"), cache, b).shape == (0, 256)


def test_step_in_a_graph(gpu):
    """A recorded step follows lengths and inputs that change in place, with
    other work between the replays."""
    rng = np.random.default_rng(2)
    layer, _, _ = build(gpu, rng, 256, 4, 2, 64)
    cache, _ = empty_cache(gpu, 8, 2, 64, 32)
    table = np.arange(8, dtype=np.int32).reshape(2, 4)
    lens = dev(np.array([40, 7], np.int32))
    b = gpu.KVBatch(dev(table), lens, max_len=128)
    x = dev(rng.normal(0, 1, (2, 256)).astype(np.float16))
    prompt = dev(rng.normal(0, 1, (45, 256)).astype(np.float16))
    _, first = batches(gpu, table, [39, 6], [39, 6], 128)
    layer(prompt, cache, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, cache, b)
        layer(x, cache, b)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = layer(x, cache, b)
    for step in range(4):
        x.copy_(dev(rng.normal(0, 1, (2, 256)).astype(np.float16)))
        lens += step > 0
        g.replay()
        got = host(y)
        again = host(layer(x, cache, b))     # storing the same tokens changes nothing
        assert np.array_equal(got, again)
        torch.cuda.synchronize()
