"""How lists of chosen pages are split, as the workspace's size tells (no GPU)."""

import pytest

import int8_quantized_matmul_absmax_amd as i8
from tests.test_kv_cache_host import batch, cache


def splits(tokens, kv_heads, group, dim, pages, page=64):
    """Of `tokens` lists a head over sequences of as many tokens as they list."""
    lib = i8.ensure_built()
    c = cache(num_pages=1 << 16, kv_heads=kv_heads, head_dim=dim, page_tokens=page)
    b = batch(num_seqs=tokens, cu_tokens=None, total_tokens=tokens, max_tokens=1, max_pages=pages,
              max_len=pages * page)
    need = lib.int8_kv_cache_attention_pages_workspace_bytes(c, b, kv_heads * group, pages)
    rows = tokens * kv_heads * group
    assert need % (4 * rows) == 0
    return (need // (4 * rows) - 1) // (dim + 2) if need else 1


@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("pages", [128, 1000, 8192])
@pytest.mark.parametrize("blocks", [1, 2, 100, 128, 200, 256, 257, 320, 511, 512, 513, 1000, 1023, 1024, 2000])
def test_no_more_splits_than_are_resident(dim, pages, blocks):
    """Two blocks a compute unit, of 256 features one."""
    resident = 256 if dim == 256 else 512
    for tokens, kv_heads, group in ((blocks, 1, 4), (blocks, 1, 9)):
        n = splits(tokens, kv_heads, group, dim, pages)
        assert n == 1 or n * blocks <= resident
        if 2 * blocks <= resident:
            assert n > 1, (blocks, n)


def test_short_lists_are_whole():
    assert splits(1, 1, 4, 128, 8) == 1 and splits(1, 1, 4, 128, 9) > 1
    assert splits(1, 1, 4, 256, 4) == 1 and splits(1, 1, 4, 256, 5) > 1
