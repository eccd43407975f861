"""Sizes past what one launch takes are refused by the checks, and those up to it are not
(no GPU: what passes the checks finds no device)."""

import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib
from tests.test_kv_cache_host import batch, cache
from tests.test_kv_sparse_host import call_attention, call_means, call_select


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    return i8.ensure_built()


@pytest.mark.parametrize("pages", [100, 8200])
@pytest.mark.parametrize("heads,tokens", [(1, (1 << 24) - 1), (32, (1 << 19) - 1), (32, 131073), (5, 3355443)])
def test_choice(lib, pages, heads, tokens):
    c = cache(kv_heads=heads, page_tokens=16)
    sizes = dict(max_tokens=4, max_pages=pages, max_len=1 << 20)
    assert call_select(lib, c, batch(total_tokens=tokens, **sizes), heads=heads) == _lib.I8MM_ENODEVICE
    if (tokens + 1) * heads > (1 << 24) - 1:
        assert call_select(lib, c, batch(total_tokens=tokens + 1, **sizes), heads=heads) == _lib.I8MM_EINVAL
        assert b"2^24" in lib.i8mm_last_error()
    none = batch(total_tokens=(1 << 24) + 1, **dict(sizes, max_tokens=0))
    assert call_select(lib, c, none, heads=heads) == _lib.I8MM_ENODEVICE


def test_attention(lib):
    """Up to eight query heads a key/value head four tokens a block, else one and 16 heads."""
    for heads, q_heads, most in ((1, 1, (1 << 26) - 4), (4, 32, (1 << 24) - 4), (1, 9, (1 << 24) - 1),
                                 (1, 17, (1 << 23) - 1), (2, 64, (1 << 22) - 1)):
        c = cache(kv_heads=heads, page_tokens=16)
        for tokens, status in ((most, _lib.I8MM_ENODEVICE), (most + 1, _lib.I8MM_EINVAL)):
            b = batch(total_tokens=tokens, max_pages=100, max_len=1 << 20)
            assert call_attention(lib, c, b, heads=q_heads) == status, (heads, q_heads, tokens)
        none = batch(total_tokens=most + 1, max_tokens=0, max_pages=100, max_len=1 << 20)
        assert call_attention(lib, c, none, heads=q_heads) == _lib.I8MM_ENODEVICE


def test_means(lib):
    for dim, parts in ((64, 1), (80, 2), (256, 4)):
        pages = ((1 << 26) - 4) // (32 * parts)          # a sequence's new tokens fill all but one
        c = cache(kv_heads=32, page_tokens=16, head_dim=dim)
        for more, status in ((0, _lib.I8MM_ENODEVICE), (1, _lib.I8MM_EINVAL)):
            n = 16 * (pages - 1 + more) - 14
            b = batch(total_tokens=n, max_tokens=n, max_pages=1 << 26, max_len=1 << 20)
            assert call_means(lib, c, b) == status, (dim, more)
