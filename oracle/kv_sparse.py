"""Plain numpy reference of attention over chosen pages of the 8-bit key/value cache,
shared with no GPU code: mean keys, the choice of pages, and the attention, all in
binary64 from the stored codes. Caches and batches as in oracle/kv_cache.py."""

import numpy as np

from oracle import kv_cache as C


def page_means(cache, means, batch):
    """Changes means fp16 [pages, heads, D] in place."""
    table, lens, counts = batch
    pages, _, slots = cache["k_absmax"].shape
    size = slots * C.BLOCK
    for b, n in enumerate(counts):
        length = int(lens[b])
        for j in range(max(length - n, 0) // size, -(-length // size)) if n > 0 else ():
            if j >= len(table[b]) or not 0 <= table[b][j] < pages:
                continue
            rows = [C.values64(cache, "k", table[b], t)
                    for t in range(j * size, min(length, (j + 1) * size))]
            with np.errstate(over="ignore", invalid="ignore"):
                mean = np.sum(rows, axis=0) / len(rows)
                means[table[b][j]] = mean.astype(np.float32).astype(np.float16)


def queries(q, pos, cos, sin, interleaved):
    """q fp16 [heads, D] rotated in binary64."""
    q = q.astype(np.float64)
    return C.rotate(q, pos, None if cos is None else cos.astype(np.float64),
                    None if sin is None else sin.astype(np.float64), interleaved)


def select_pages(cache, means, q, batch, count, first=1, recent=1, cos=None, sin=None,
                 interleaved=False):
    """-> (int32 [tokens, heads, count], the least gap between the scores of a page
    that is chosen by its score and one that is not)."""
    table, lens, counts = batch
    pages, heads, slots = cache["k_absmax"].shape
    size = slots * C.BLOCK
    out = np.full((q.shape[0], heads, count), -1, np.int32)
    group = q.shape[1] // heads
    row, gap = 0, np.inf
    for b, n in enumerate(counts):
        for i in range(n):
            pos = int(lens[b]) - n + i
            if pos >= 0:
                x = queries(q[row], pos, cos, sin, interleaved)
                seen = pos // size + 1
                for h in range(heads):
                    sure = [j for j in range(seen) if j < first or j >= seen - recent]
                    rest = []
                    for j in range(seen):
                        if j in sure:
                            continue
                        page = table[b][j]
                        score = -np.inf
                        if 0 <= page < pages:
                            with np.errstate(invalid="ignore"):
                                score = float(x[h * group:(h + 1) * group].sum(axis=0)
                                              @ means[page, h].astype(np.float64))
                        rest.append((-np.inf if np.isnan(score) else score, -j))
                    rest.sort(reverse=True)
                    if seen <= count:
                        picked = list(range(seen))
                    else:
                        want = count - len(sure)
                        picked = sorted(sure + [-j for _, j in rest[:want]])
                        if 0 < want < len(rest) and rest[want - 1][0] != rest[want][0]:
                            gap = min(gap, rest[want - 1][0] - rest[want][0])
                    out[row, h, :len(picked)] = picked
            row += 1
    return out, gap


def attention_pages(cache, q, batch, chosen, cos=None, sin=None, interleaved=False, scale=None):
    """-> (O, bound) fp64 [tokens, q_heads, D]; the bound as oracle/kv_cache.py's, the
    weights in two parts of fp16 (22 bits)."""
    table, lens, counts = batch
    pages, kv_heads, slots = cache["k_absmax"].shape
    size = slots * C.BLOCK
    heads, d = q.shape[1:]
    group = heads // kv_heads
    scale = 1.0 / np.sqrt(d) if scale is None else float(scale)
    out = np.zeros(q.shape, np.float64)
    bound = np.full(q.shape, 2.0 ** -24)
    row = 0
    for b, n in enumerate(counts):
        length = int(lens[b])
        ks = [C.values(cache, "k", table[b], t) for t in range(length)]
        vs = [C.values(cache, "v", table[b], t) for t in range(length)]
        for i in range(n):
            pos = length - n + i
            for h in range(heads if pos >= 0 else 0):
                seen = [t for j in chosen[row, h // group] if j >= 0
                        for t in range(int(j) * size, min(int(j) * size + size, pos + 1))
                        if ks[t] is not None]
                if not seen:
                    continue
                x = C.rotate(q[row].astype(np.float32), pos, cos, sin, interleaved)
                x = x[h].astype(np.float64)
                kh = np.array([ks[t][h // group] for t in seen], np.float64)
                vh = np.array([vs[t][h // group] for t in seen], np.float64)
                z = kh @ x * scale
                p = np.exp(z - z.max())
                total = p.sum()
                o = p @ vh / total
                spread = p @ np.abs(vh) / total + np.abs(o)
                err = scale * np.abs(x).max() / 32512 * np.abs(kh).sum(axis=1).max()
                err += 2.0 ** -20 * (scale * (np.abs(kh) @ np.abs(x)).max() + np.abs(z).max())
                out[row, h] = o
                bound[row, h] += (np.expm1(2 * err) + 2.0 ** -20 + len(seen) * 2.0 ** -23) * spread \
                    + 2.0 ** -11 * np.abs(o) + len(seen) * 2.0 ** -25 * np.abs(vh).max()
            row += 1
    return out, bound
