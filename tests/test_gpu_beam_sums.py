"""The sums of beam selection against 64 bits, on rows that make them as hard as they
get: maxima that rise with every part of a row, long flat rows, one word far above."""

import numpy as np
import pytest
import torch

from tests.gpu_helpers import dev, host, note

pytestmark = pytest.mark.gpu

# What the header says a row's sum is within, relative to itself: of its logarithm, and
# so of a value, as much absolutely.
SUM = 2.0 ** -16


def rows(rng, vocab, half):
    at = np.arange(vocab)
    part = 8192 if half else 4096
    lane = (at // (8 if half else 4)) % 64
    kinds = [0.3 * (at // part), 0.01 * (at // part), -0.01 * (at // part),
             (at // part + 0.1 * lane) * 0.2, at * (16.0 / vocab), np.zeros(vocab),
             np.where(at == vocab // 3, 13.1, 0.0), rng.normal(0, 1, vocab) - 20,
             rng.normal(0, 4, vocab), -np.log1p(at), 1000.0 + rng.random(vocab)]
    return np.stack(kinds).astype(np.float16 if half else np.float32)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("vocab,copies", [(1 << 20, 1), (1 << 18, 100), (50257, 30), (1 << 24, 1), (4099, 1)])
def test_sums(gpu, half, vocab, copies):
    note("sums %s" % ((half, vocab, copies),))
    x = dev(rows(np.random.default_rng(vocab), vocab, half))
    wide = x.double()
    top = wide.amax(dim=1)
    total = torch.log(torch.exp(wide - top[:, None]).sum(dim=1))
    del wide
    # scores that leave a value near 0, whose own rounding is then nothing
    scores = total.float()
    want = host(scores.double() - total)
    n = x.shape[0]
    many = x.unsqueeze(1).expand(n, copies, vocab).reshape(n * copies, 1, vocab)
    got = gpu.beam_select(many, scores.repeat_interleave(copies).view(-1, 1), count=1)[0]
    off = np.abs(host(got).reshape(n, copies).astype(np.float64) - want[:, None]).max(axis=1)
    print("largest error of a logarithm, 2^-24:", np.round(off * 2 ** 24, 1).tolist())
    assert (off <= SUM).all(), off
