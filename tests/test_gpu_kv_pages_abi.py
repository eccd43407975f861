"""The step of the page tables that gives no lengths for a batch, by its C entry point:
what the other one gives."""

import pytest
import torch

from oracle import kv_pages as R
from tests.gpu_helpers import host, note
from tests.test_gpu_kv_pages import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [30, 20000])
def test_step_without_lengths_for_the_batch(gpu, pages):
    """In one launch and in several."""
    lib = gpu.load_library()
    table, lens, parents, new = [[5, 1, 7], [5, 2, -1]], [47, 20], [0, 0, 1, -1, 1], [3, 1, 1, 20, 0]
    note("step by the C entry, %d pages" % pages)
    need = lib.i8mm_kv_pages_workspace_bytes(5, 3, pages)
    assert (need > 0) == (pages == 20000)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    t, n, p, w = ints(table), ints(lens), ints(parents), ints(new)
    out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((5, 3), (5,), (5, 3), (2,))]
    status = lib.i8mm_kv_pages_step(
        t.data_ptr(), n.data_ptr(), 2, 3, p.data_ptr(), None, w.data_ptr(), 0, 5, pages, 16,
        *[x.data_ptr() for x in out], ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    want = R.step(table, lens, parents, new, None, pages, 16, 3)
    assert host(out[0]).tolist() == want[0] and host(out[1]).tolist() == want[1]
    assert host(out[2]).tolist() == [list(c) for c in want[2]] + [[-1] * 3] * (5 - len(want[2]))
    assert host(out[3]).tolist() == [len(want[2]), want[3]]
    batch = gpu.ops.kv_pages_step(t, n, p, pages, 16, w, batch=True)
    for a, b in zip(out, batch):
        assert torch.equal(a, b)
    assert host(batch[4]).tolist() == [0, 48, 21, 20, 0] and host(batch[5]).tolist() == [1]
