"""Calls near what one launch takes."""

import pytest
import torch

from tests.gpu_helpers import host, note

pytestmark = pytest.mark.gpu


def test_choice_of_more_lists_than_a_launch_of_large_blocks_takes(gpu):
    """More than 2^22 lists, with more than 4096 pages to choose from: blocks of 1024
    threads would be too many. Nearly all of the rows belong to no sequence; those that
    do get what they get in a small call."""
    heads, page, tokens, width = 32, 16, 131073, 4200
    note("choice, %d lists" % (heads * tokens))
    gen = torch.Generator(device="cuda").manual_seed(5)
    c = gpu.Int8KVCache(300, heads, 64, page, page_means=True)
    c.k_means.copy_(torch.randn(c.k_means.shape, device="cuda", generator=gen))
    table = torch.randint(0, 300, (2, width), dtype=torch.int32, device="cuda", generator=gen)
    lens = torch.tensor([67000, 40], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    q = torch.zeros((tokens, heads, 64), dtype=torch.float16, device="cuda")
    q[:5] = torch.randn((5, heads, 64), device="cuda", generator=gen)
    large = gpu.KVBatch(table, lens, cu, total_tokens=tokens, max_tokens=4)
    small = gpu.KVBatch(table, lens, cu, total_tokens=5)
    got = c.select_pages(q, large, 6)
    want = c.select_pages(q[:5], small, 6)
    assert torch.equal(got[:5], want) and bool((got[5:] == -1).all())
    assert (host(want)[:3] >= 0).all() and host(want)[3, 0].tolist() == [0, 1, 2, -1, -1, -1]
