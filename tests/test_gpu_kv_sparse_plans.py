"""Attention over chosen pages where lists are long and stay whole, or nearly so."""

import numpy as np
import pytest

from tests.test_gpu_kv_sparse import check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,length,count,heads,kv,dim,page", [
    (257, 5000, 310, 2, 1, 64, 16),      # whole
    (100, 9000, 560, 4, 2, 64, 16),      # in two
    (20, 9001, 280, 72, 8, 128, 32),     # in three, nine heads a list
    (129, 6000, 125, 3, 1, 256, 48)])
def test_long_lists_of_many_tokens(gpu, tokens, length, count, heads, kv, dim, page):
    check_attention(gpu, np.random.default_rng(length), [length], [tokens], heads, kv, dim, page, count)
