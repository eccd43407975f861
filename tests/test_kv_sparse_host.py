"""Host-side checks of attention over chosen pages: refusals of the C ABI and of the
binding (no GPU, no compute calls), and pins of the numpy reference."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib, ops
from oracle import kv_cache as C
from oracle import kv_sparse as R
from tests import test_kv_cache_host as T
from tests.test_kv_cache_host import A, MIS, ODD, batch, cache, rotary


@pytest.fixture(scope="module")
def lib():
    return i8.ensure_built()


def call_means(lib, c, b, means=A):
    return lib.int8_kv_cache_page_means(c, b, means, None)


def call_select(lib, c, b, r=None, q=A, strides=(256, 64), heads=4, means=A, count=3, first=1, recent=1,
                out=A):
    return lib.int8_kv_cache_select_pages(q, strides[0], strides[1], heads, c, means, b, r, count, first,
                                          recent, out, None)


def call_attention(lib, c, b, r=None, q=A, strides=(256, 64), heads=4, pages=A, count=3, scale=0.125,
                   out=A, ws=A, wn=1 << 40):
    return lib.int8_kv_cache_attention_pages(q, strides[0], strides[1], heads, c, b, r, pages, count,
                                             scale, out, ws, wn, None)


@pytest.mark.parametrize("ck,bk,status", T.BAD_SIZES + T.BAD_POINTERS)
def test_refused_cache_or_batch(lib, ck, bk, status):
    c, b = cache(**ck), batch(**bk)
    assert call_means(lib, c, b) == status
    assert lib.i8mm_last_error().startswith(b"int8_kv_cache_page_means: ")
    assert call_select(lib, c, b) == status
    assert lib.i8mm_last_error().startswith(b"int8_kv_cache_select_pages: ")
    assert call_attention(lib, c, b) == status
    assert lib.i8mm_last_error().startswith(b"int8_kv_cache_attention_pages: ")


@pytest.mark.parametrize("rk,status", [
    (dict(dim=0), _lib.I8MM_EINVAL), (dict(dim=80), _lib.I8MM_EINVAL),
    (dict(positions=255), _lib.I8MM_EINVAL), (dict(cos=None), _lib.I8MM_EINVAL),
    (dict(sin=MIS), _lib.I8MM_EALIGN)])
def test_refused_rotary(lib, rk, status):
    assert call_select(lib, cache(), batch(), rotary(**rk)) == status
    assert call_attention(lib, cache(), batch(), rotary(**rk)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), _lib.I8MM_EINVAL), (dict(q=MIS), _lib.I8MM_EALIGN),
    (dict(strides=(-8, 64)), _lib.I8MM_EINVAL), (dict(strides=(256, 12)), _lib.I8MM_EALIGN),
    (dict(heads=3), _lib.I8MM_EINVAL), (dict(heads=0), _lib.I8MM_EINVAL),
    (dict(count=0), _lib.I8MM_EINVAL), (dict(count=-1), _lib.I8MM_EINVAL),
    (dict(count=(1 << 24) + 1), _lib.I8MM_EINVAL), (dict(count=1 << 62), _lib.I8MM_EINVAL),
    (dict(out=None), _lib.I8MM_EINVAL)])
def test_refused_by_both(lib, kw, status):
    assert call_select(lib, cache(), batch(), **kw) == status
    assert call_attention(lib, cache(), batch(), **kw) == status


def test_refused_choices(lib):
    for kw in (dict(first=-1), dict(recent=0), dict(first=3), dict(first=2, recent=2),
               dict(first=1 << 62, recent=1 << 62)):
        assert call_select(lib, cache(), batch(), **kw) == _lib.I8MM_EINVAL, kw
    assert call_select(lib, cache(), batch(), means=None) == _lib.I8MM_EINVAL
    assert call_select(lib, cache(), batch(), means=MIS) == _lib.I8MM_EALIGN
    assert call_select(lib, cache(), batch(), out=ODD) == _lib.I8MM_EALIGN
    assert call_means(lib, cache(), batch(), means=None) == _lib.I8MM_EINVAL
    assert call_means(lib, cache(), batch(), means=MIS) == _lib.I8MM_EALIGN
    # more pages than the choice has room for
    b = batch(max_pages=16387, max_len=1 << 30)
    assert call_select(lib, cache(), b) == _lib.I8MM_EINVAL
    assert b"16384 pages" in lib.i8mm_last_error()


def test_refused_attention(lib):
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call_attention(lib, cache(), batch(), scale=scale) == _lib.I8MM_EINVAL
    assert call_attention(lib, cache(), batch(), pages=None) == _lib.I8MM_EINVAL
    assert call_attention(lib, cache(), batch(), pages=ODD) == _lib.I8MM_EALIGN
    assert call_attention(lib, cache(), batch(), out=MIS) == _lib.I8MM_EALIGN
    c, b = cache(), batch(max_pages=1 << 12, max_len=1 << 17)
    need = lib.int8_kv_cache_attention_pages_workspace_bytes(c, b, 4, 64)
    assert need > 0
    for kw, status in ((dict(ws=None), _lib.I8MM_EWORKSPACE), (dict(wn=need - 1), _lib.I8MM_EWORKSPACE),
                       (dict(ws=A + 64), _lib.I8MM_EALIGN)):
        assert call_attention(lib, c, b, count=64, **kw) == status
    for heads, count in ((3, 64), (0, 64), (4, 0), (4, 1 << 40)):
        assert lib.int8_kv_cache_attention_pages_workspace_bytes(c, b, heads, count) == 0
    assert lib.int8_kv_cache_attention_pages_workspace_bytes(None, b, 4, 4) == 0


def test_nothing_to_do_needs_no_device(lib):
    none = dict(page_table=None, seq_lens=None, cu_tokens=None, num_seqs=0, total_tokens=0)
    assert call_means(lib, cache(), batch(**none)) == 0
    assert call_select(lib, cache(), batch(**none), q=None, out=None) == 0
    assert call_attention(lib, cache(), batch(**none), q=None, pages=None, out=None, ws=None, wn=0) == 0


def test_no_tokens_of_long_sequences(lib):
    """Nothing to split, however long the lists are."""
    for tokens in (0, 2):
        b = batch(num_seqs=tokens, total_tokens=tokens, cu_tokens=None, max_pages=5000, max_len=320000)
        need = lib.int8_kv_cache_attention_pages_workspace_bytes(cache(num_pages=9000), b, 4, 4000)
        assert (need > 0) == (tokens > 0)


def test_binding_refusals():
    class Cache:
        device, k_means, kv_heads, head_dim, ref = torch.device("cpu"), None, 2, 64, None

    class Batch:
        device, total_tokens, ref = torch.device("cpu"), 3, None
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    pages = torch.zeros((3, 2, 5), dtype=torch.int32)
    with pytest.raises(ValueError, match="mean keys"):
        ops.int8_kv_cache_page_means(Cache, Batch)
    with pytest.raises(ValueError, match="mean keys"):
        ops.int8_kv_cache_select_pages(q, Cache, Batch, 3)
    with pytest.raises(TypeError):
        ops.int8_kv_cache_attention_pages(q, pages.long(), Cache, Batch)
    with pytest.raises(ValueError):
        ops.int8_kv_cache_attention_pages(q, pages[:2], Cache, Batch)
    with pytest.raises(ValueError):
        ops.int8_kv_cache_attention_pages(q, pages[:, :1].contiguous(), Cache, Batch)
    with pytest.raises(ValueError):
        ops.int8_kv_cache_attention_pages(q, pages[:, 0].contiguous(), Cache, Batch)
    with pytest.raises(ValueError):                       # on the host
        ops.int8_kv_cache_attention_pages(q, pages, Cache, Batch)


# ------------------------------------------------------------------ reference

def test_reference_pins():
    """Every page listed in order is the dense attention; a page listed twice counts
    twice; the mean of one token is the token; the best page holds the query's key."""
    rng = np.random.default_rng(1)
    c = T.empty(4, 2, 64, 16)
    b = (np.array([[2, 0, 3]]), [41], [41])
    k, v = rng.normal(0, 1, (2, 41, 2, 64)).astype(np.float16)
    C.append(c, k, v, b)
    q = rng.normal(0, 1, (41, 4, 64)).astype(np.float16)
    every = np.broadcast_to(np.arange(3), (41, 2, 3))
    dense, _ = C.attention(c, q, b)
    got, bound = R.attention_pages(c, q, b, every)
    assert np.allclose(got, dense, atol=1e-12) and (bound > 0).all()
    twice, _ = R.attention_pages(c, q, b, every[:, :, [0, 0, 1, 1, 2, 2, 2]][:, :, :6])
    assert np.allclose(twice, dense, atol=1e-12)
    assert not R.attention_pages(c, q, b, np.full((41, 2, 2), -1))[0].any()
    means = np.zeros((4, 2, 64), np.float16)
    R.page_means(c, means, (b[0], [33], [1]))
    one = C.values(c, "k", b[0][0], 32)
    assert np.array_equal(means[3], one.astype(np.float16)) and not means[:3].any()
    R.page_means(c, means, b)
    picked, gap = R.select_pages(c, means, q[-1:] * 0 + 1, (b[0], [41], [1]), 2)
    assert picked.tolist() == [[[0, 2], [0, 2]]] and gap == np.inf
    x = (8 * means[0].astype(np.float64)).repeat(2, axis=0).astype(np.float16)
    picked, gap = R.select_pages(c, means, x[None], (b[0], [41], [1]), 2, first=0)
    assert picked.tolist() == [[[1, 2], [1, 2]]] and gap > 0
