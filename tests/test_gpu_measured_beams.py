"""Measured beam selections: their plain form, their 64-bit definition and the operator
agree on what is chosen, with fewer candidates than places too."""

import math

import numpy as np
import pytest
import torch

from oracle import beam as R
from perf import more_operators as P
from tests.gpu_helpers import host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", ["ended", "masked", "none"])
def test_fewer_candidates_than_places(gpu, monkeypatch, case):
    logits = torch.randn((1, 1, 50), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    live = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    if case == "ended":
        live.zero_()
    else:
        logits[:, :, 2 if case == "masked" else 0:] = -math.inf
    s = {"logits": logits, "scores": torch.full((1, 1), -3.0, device="cuda"), "live": live, "eos": 2,
         "case": dict(op="beam", batch=1, beams=1, vocab=50, count=4, half=False)}
    want = R.select(host(logits), host(s["scores"]), host(live), 2, 4)
    found = {"ended": 1, "masked": 2, "none": 0}[case]
    assert np.isfinite(want[0]).sum() == found
    exact = P._exact_beam(s["case"], s)
    outs = [exact]
    for own in (False, True):
        monkeypatch.setattr(P, "own", own)
        outs.append(P.run(s))
    for out in outs:
        for got, expected in zip(out[1:], want[1:4]):
            assert np.array_equal(host(got), expected)
        got = host(out[0]).astype(np.float64)
        assert np.array_equal(np.isfinite(got), np.isfinite(want[0]))
        # a row's sum within 2^-16 of itself, and a rounding to 32 bits of values below 16
        assert np.allclose(got[0, :found], want[0][0, :found], rtol=0, atol=2.0 ** -16 + 2.0 ** -21)
