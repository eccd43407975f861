"""Plain numpy reference of the paged 8-bit key/value cache, shared with no GPU
code.

Rotation, absmax, codes and stored values are one binary32 operation at a time,
as the C ABI states them, so they are compared bit for bit; attention is in
binary64 from the stored codes and absmaxes.

A cache is a dict of k_codes, v_codes [pages, heads, slots, D/16, 16, 16] int8
and k_absmax, v_absmax [pages, heads, slots] fp32. A batch is (page_table,
seq_lens, counts): counts[b] new tokens of sequence b are its last.
"""

import numpy as np

BLOCK = 16
TINY = np.float32(2.0) ** np.float32(-119)
F = np.float32


def rotate(x, pos, cos, sin, interleaved):
    """x fp32 [heads, D] at position pos."""
    if cos is None:
        return x
    y = x.copy()
    c, s = cos[pos], sin[pos]
    half = c.shape[0]
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + 1 if interleaved else i1 + half
    y[:, i1] = x[:, i1] * c - x[:, i2] * s
    y[:, i2] = x[:, i2] * c + x[:, i1] * s
    return y


def place(cache, table_row, t):
    """(page, slot, row) of token t, or None when its page is absent."""
    pages, _, slots = cache["k_absmax"].shape
    p = t // (slots * BLOCK)
    if p >= len(table_row) or not 0 <= table_row[p] < pages:
        return None
    return int(table_row[p]), t // BLOCK % slots, t % BLOCK


def get_rows(cache, which, page, slot):
    """Codes of a block as [heads, 16 tokens, D]."""
    c = cache[which + "_codes"][page, :, slot]              # [heads, D/16, 16, 16]
    c = c.transpose(0, 2, 1, 3) if which == "k" else c.transpose(0, 3, 1, 2)
    return c.reshape(c.shape[0], BLOCK, -1)


def set_rows(cache, which, page, slot, rows):
    h, _, d = rows.shape
    r = rows.reshape(h, BLOCK, d // 16, 16)
    r = r.transpose(0, 2, 1, 3) if which == "k" else r.transpose(0, 2, 3, 1)
    cache[which + "_codes"][page, :, slot] = r


def append(cache, k, v, batch, cos=None, sin=None, interleaved=False):
    """k, v fp16 [tokens, heads, D]; changes the cache in place."""
    table, lens, counts = batch
    row0 = 0
    for b, n in enumerate(counts):
        first = int(lens[b]) - n
        for blk in range(max(first, 0) // BLOCK, -(-int(lens[b]) // BLOCK)):
            at = place(cache, table[b], blk * BLOCK)
            if at is None or n == 0:
                continue
            page, slot, _ = at
            r0 = max(first - blk * BLOCK, 0)
            r1 = min(BLOCK, int(lens[b]) - blk * BLOCK)
            for which, src in (("k", k), ("v", v)):
                new = src[row0 + blk * BLOCK + r0 - first:row0 + blk * BLOCK + r1 - first]
                new = new.astype(F)
                if which == "k":
                    new = np.stack([rotate(x, blk * BLOCK + r0 + i, cos, sin, interleaved)
                                    for i, x in enumerate(new)])
                top = np.abs(new).max(axis=(0, 2))
                old = np.abs(cache[which + "_absmax"][page, :, slot]) if r0 else np.zeros_like(top)
                a = np.maximum(top, old)
                a = np.where(a <= TINY, F(0), a).astype(F)
                with np.errstate(divide="ignore", invalid="ignore"):
                    s = np.where(a > 0, F(127) / a, F(0)).astype(F)
                    ratio = np.where(a > 0, old / a, F(0)).astype(F)
                rows = get_rows(cache, which, page, slot).copy()
                grown = a != old
                kept = np.rint(rows[:, :r0].astype(F) * ratio[:, None, None])
                rows[:, :r0] = np.where(grown[:, None, None], kept, rows[:, :r0])
                rows[:, r0:] = 0
                rows[:, r0:r1] = np.rint(new.transpose(1, 0, 2) * s[:, None, None])
                set_rows(cache, which, page, slot, rows)
                cache[which + "_absmax"][page, :, slot] = a
        row0 += n


def values(cache, which, table_row, t):
    """Stored values [heads, D] of token t in fp32, or None when absent."""
    at = place(cache, table_row, t)
    if at is None:
        return None
    page, slot, row = at
    step = cache[which + "_absmax"][page, :, slot] / F(127)
    return get_rows(cache, which, page, slot)[:, row].astype(F) * step[:, None]


def read(cache, batch):
    """Keys and values of the batch's tokens, fp16 [tokens, heads, D]."""
    table, lens, counts = batch
    _, heads, _, tiles = cache["k_codes"].shape[:4]
    outs = []
    for which in "kv":
        rows = []
        for b, n in enumerate(counts):
            for t in range(int(lens[b]) - n, int(lens[b])):
                x = values(cache, which, table[b], t) if t >= 0 else None
                rows.append(np.zeros((heads, tiles * 16), F) if x is None else x)
        outs.append(np.array(rows, F).reshape(len(rows), heads, tiles * 16).astype(np.float16))
    return outs


def attention(cache, q, batch, cos=None, sin=None, interleaved=False, scale=None, causal=True,
              window=0, slopes=None):
    """q fp16 [tokens, q_heads, D] -> (O, bound) fp64 [tokens, q_heads, D].

    bound: what a result may be off by when the query is rounded to 15 bits over
    its row's absmax, the weights to fp16 against the row's maximum, the output
    to fp16, and everything else is binary32. A change of the logits of at most
    e changes O by at most (exp(2 e) - 1) times sum(p |v|) + |O|."""
    table, lens, counts = batch
    heads = q.shape[1]
    group = heads // cache["k_codes"].shape[1]
    d = q.shape[2]
    scale = 1.0 / np.sqrt(d) if scale is None else float(scale)
    out = np.zeros(q.shape, np.float64)
    bound = np.full(q.shape, 2.0 ** -24)
    row = 0
    for b, n in enumerate(counts):
        length = int(lens[b])
        ks = [values(cache, "k", table[b], t) for t in range(length)]
        vs = [values(cache, "v", table[b], t) for t in range(length)]
        for i in range(n):
            pos = length - n + i
            seen = [t for t in range(length) if ks[t] is not None and pos >= 0
                    and (t <= pos or not causal) and (window == 0 or t > pos - window)]
            if seen:
                x = rotate(q[row].astype(F), pos, cos, sin, interleaved).astype(np.float64)
                K = np.array([ks[t] for t in seen], np.float64)      # [T, kv_heads, D]
                V = np.array([vs[t] for t in seen], np.float64)
                for h in range(heads):
                    kh, vh = K[:, h // group], V[:, h // group]
                    z = kh @ x[h] * scale
                    if slopes is not None:
                        z = z - float(slopes[h]) * (pos - np.array(seen, np.float64))
                    p = np.exp(z - z.max())
                    L = p.sum()
                    o = p @ vh / L
                    spread = p @ np.abs(vh) / L + np.abs(o)
                    err = scale * np.abs(x[h]).max() / 32512 * np.abs(kh).sum(axis=1).max()
                    err += 2.0 ** -20 * (scale * (np.abs(kh) @ np.abs(x[h])).max()
                                         + np.abs(z).max())
                    tail = len(seen) * 2.0 ** -25 * np.abs(vh).max()
                    out[row, h] = o
                    bound[row, h] += (np.expm1(2 * err) + 2.0 ** -11 + len(seen) * 2.0 ** -23) \
                        * spread + 2.0 ** -11 * np.abs(o) + tail
            row += 1
    return out, bound
