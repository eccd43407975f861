"""Plain numpy reference of a beam search's selection, in binary64, shared with no
GPU code."""

import numpy as np


def select(logits, scores, live, eos, count):
    """logits [batch, beams, vocab], scores and live [batch, beams] (live None: all)
    -> (scores fp64, tokens, parents, live, gap), each [batch, count] but gap
    [batch]: the least distance between a chosen value and the next candidate of
    another beam, which is how far values may be off without another choice."""
    batch, beams, vocab = logits.shape
    out = (np.full((batch, count), -np.inf), np.full((batch, count), -1, np.int64),
           np.full((batch, count), -1, np.int64), np.zeros((batch, count), np.int64))
    gaps = np.full(batch, np.inf)
    for b in range(batch):
        found = []
        for i in range(beams):
            s = float(scores[b, i])
            if not np.isfinite(s):
                continue
            if live is not None and live[b, i] == 0:
                found.append((-s, i, max(eos, 0), eos))
                continue
            x = logits[b, i].astype(np.float64)
            if np.isnan(x).any() or not x.size or x.max() in (np.inf, -np.inf):
                continue
            base = s - x.max() - np.log(np.exp(x - x.max()).sum())
            # the best `count` words and all that equal the last of them
            edge = np.sort(x)[::-1][min(count, vocab) - 1]
            for v in np.flatnonzero((x >= edge) & (x > -np.inf)):
                found.append((-(base + x[v]), i, int(v), int(v)))
        found.sort(key=lambda c: c[:3])
        for j, (value, i, _, token) in enumerate(found[:count]):
            for o, x in zip(out, (-value, token, b * beams + i,
                                  int((live is None or live[b, i] != 0) and token != eos))):
                o[b, j] = x
        for a, c in zip(found[:count], found[1:count + 1]):
            if a[1] != c[1]:
                gaps[b] = min(gaps[b], c[0] - a[0])
    return out + (gaps,)
