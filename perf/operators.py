"""Measured cases of the paged 8-bit key/value cache: appending keys and values
(position rotation and quantization on the way), attention over the cache, and
reading cached values back.

The cache holds int8 codes in 16 x 16 byte tiles, one absmax for each block of
16 tokens and head. Page p, head h, block s, tile c:
  k_codes[p, h, s, c, t, e]  key code of token 16 s + t, feature 16 c + e
  v_codes[p, h, s, c, e, t]  value code of the same token and feature
  k_absmax[p, h, s], v_absmax[p, h, s]; a code stands for code * absmax / 127.

A sequence's new tokens are its last ones: with n new tokens of length L they
have the positions L - n .. L - 1.
"""

import math
import random

import torch

own = False

BLOCK = 16


# --------------------------------------------------------------------- cases

def _case(op, batch, new, shortest, longest, heads, kv_heads, dim, page, rotary=0,
          interleaved=False, alibi=False, window=0, ragged_new=False, name=None):
    case = {"op": op, "batch": batch, "new": new, "shortest": shortest, "longest": longest,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "rotary": rotary,
            "interleaved": interleaved, "alibi": alibi, "window": window,
            "ragged_new": ragged_new}
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # one conversation's next token early on, at the hidden size 4096 of the
        # decode workload (32 heads of 128): launch latency
        _case("attention", 1, 1, 61, 61, 32, 32, 128, 64, rotary=128,
              name="attention_one_token_short"),
        # the decode batch of 16 tokens, hidden size 4096, conversations of every length
        _case("attention", 16, 1, 1, 4096, 32, 32, 128, 64, rotary=128,
              name="attention_16_ragged"),
        # one token at the end of a very long document, grouped heads: the
        # long axis has to be split to fill the card
        _case("attention", 1, 1, 131071, 131071, 32, 8, 128, 128, rotary=128,
              name="attention_one_token_long"),
        # a full serving batch with grouped heads and small pages: cache bandwidth
        _case("attention", 64, 1, 100, 8192, 64, 8, 128, 16, rotary=64, interleaved=True,
              name="attention_64_grouped"),
        # a scheduler's step that mixes prompt chunks with single tokens over
        # cached prefixes, linear position biases in place of a rotation
        _case("attention", 8, 512, 1, 8191, 32, 8, 64, 48, alibi=True, ragged_new=True,
              name="attention_chunks"),
        # a prompt of 4096 tokens at hidden size 12288 (96 heads of 128): compute
        _case("attention", 1, 4096, 4096, 4096, 96, 96, 128, 64, rotary=128,
              name="attention_prompt_wide"),
        # one new token of one conversation: launch latency
        _case("append", 1, 1, 1000, 1000, 32, 32, 128, 64, rotary=128,
              name="append_one_token"),
        # the decode batch of 16 tokens, each in the middle of some block
        _case("append", 16, 1, 1, 4096, 32, 32, 128, 64, rotary=128,
              name="append_16_ragged"),
        # a scheduler's step of ragged prompt chunks, grouped heads, 80 features a head
        _case("append", 8, 512, 1, 8191, 32, 8, 80, 48, rotary=32, interleaved=True,
              ragged_new=True, name="append_chunks"),
        # a prompt of 4096 tokens at hidden size 12288: bandwidth
        _case("append", 1, 4096, 4096, 4096, 96, 96, 128, 64, rotary=128,
              name="append_prompt_wide"),
        # one conversation's cache taken out in 16 bits, to move or inspect it
        _case("read", 1, 1000, 1000, 1000, 32, 8, 128, 64, name="read_one"),
        # the caches of a batch taken out in 16 bits, odd lengths
        _case("read", 12, 8191, 1, 8191, 64, 16, 128, 16, ragged_new=True, name="read_batch"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    largest = {op: max(_cost(c) for c in listed() if c["op"] == op)
               for op in ("attention", "append", "read")}
    op = rng.choice(("attention", "attention", "append", "read"))
    while True:
        dim = rng.choice((64, 80, 96, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 5, 8, 16, 32))
        group = rng.choice((1, 1, 2, 3, 4, 6, 8))
        positions = rng.choice(("rotary", "partial", "alibi", "none"))
        rotary = {"rotary": dim, "partial": dim // 32 * 16}.get(positions, 0)
        batch = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, 32768)
        new = 1
        if op == "read":
            new = longest
        elif rng.random() < 0.5:
            new = _log_int(rng, 1, min(longest, 4096))
        case = _case(op, batch, new, rng.choice((1, longest)), longest, kv_heads * group,
                     kv_heads, dim, 16 * rng.randint(1, 8), rotary, rng.random() < 0.3,
                     op == "attention" and positions == "alibi",
                     _log_int(rng, 16, 8192) if op == "attention" and rng.random() < 0.25 else 0,
                     rng.random() < 0.5)
        # the plain form's padded sizes bound it too
        if _cost(case) <= largest[op] and batch * longest * kv_heads * dim <= 1 << 28:
            return case


def _sizes(case):
    """(new tokens, length) of each sequence; the first is the longest."""
    rng = random.Random(case["batch"] * 1000003 + case["longest"] * 101 + case["new"])
    sizes = []
    for i in range(case["batch"]):
        n = case["new"] if i == 0 or not case["ragged_new"] else rng.randint(1, case["new"])
        low = max(n, min(case["shortest"], case["longest"]))
        length = case["longest"] if i == 0 else rng.randint(low, case["longest"])
        sizes.append((n, length if case["op"] != "read" else n))
    return sizes


def _visible(n, length, window):
    """Pairs of a new token and a cached token that it sees."""
    total = n * length - n * (n - 1) // 2
    if window:
        for p in range(length - n, length):
            total -= max(0, p + 1 - window)
    return total


def work(case):
    sizes = _sizes(case)
    tokens = sum(n for n, _ in sizes)
    d, hkv, h = case["dim"], case["kv_heads"], case["heads"]
    table = 4 * case["rotary"] * tokens if case["rotary"] else 0
    if case["op"] == "attention":
        cached = 0
        for n, length in sizes:
            first = max(0, length - n + 1 - case["window"]) if case["window"] else 0
            cached += length - first
        blocks = cached / BLOCK
        return {"bytes": 2 * cached * hkv * d + 8 * blocks * hkv + 4 * tokens * h * d + table,
                "flops": 4 * d * h * sum(_visible(n, l, case["window"]) for n, l in sizes)}
    if case["op"] == "append":
        old = sum((l - n) % BLOCK for n, l in sizes)
        # new keys and values in 16 bits, their codes, the old codes of the
        # blocks they share, and the values of these blocks in 16 bits
        return {"bytes": (4 + 2) * tokens * hkv * d + 2 * old * hkv * d + table
                + 4 * (tokens + old) * hkv * d,
                "flops": 10 * (tokens + old) * hkv * d}
    return {"bytes": 6 * tokens * hkv * d, "flops": 2 * tokens * hkv * d}


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / 1e15


# -------------------------------------------------------------------- inputs

def _values(shape, gen, channels):
    """Keys or values as projections give them: a level for each token and, for
    keys, a few features much larger than the rest."""
    x = torch.randn(shape, device="cuda", generator=gen)
    x *= torch.exp(0.4 * torch.randn(shape[:-1] + (1,), device="cuda", generator=gen))
    if channels:
        gain = torch.ones(shape[-1], device="cuda")
        gain[torch.randperm(shape[-1], device="cuda", generator=gen)[:4]] = 4.0
        x *= gain
    return x


def _filled(pages, case, gen, keys):
    """Codes and absmax of a cache whose every block holds tokens."""
    hkv, d, slots = case["kv_heads"], case["dim"], case["page"] // BLOCK
    x = _values((pages, hkv, slots, BLOCK, d), gen, keys)
    absmax = x.abs().amax(dim=(3, 4))
    codes = torch.round(x * (127.0 / absmax)[..., None, None]).to(torch.int8)
    codes = codes.view(pages, hkv, slots, BLOCK, d // 16, 16)
    codes = codes.permute(0, 1, 2, 4, 3, 5) if keys else codes.permute(0, 1, 2, 4, 5, 3)
    return codes.contiguous(), absmax


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    sizes = _sizes(case)
    page, hkv, d = case["page"], case["kv_heads"], case["dim"]
    counts = [-(-length // page) for _, length in sizes]
    pages = sum(counts) + 2
    order = torch.randperm(pages, device="cuda", generator=gen).tolist()
    width = max(counts)
    table, at = [], 0
    for c in counts:
        table.append(order[at:at + c] + [-1] * (width - c))
        at += c
    ints = dict(dtype=torch.int32, device="cuda")
    tokens = sum(n for n, _ in sizes)
    starts = [0]
    for n, _ in sizes:
        starts.append(starts[-1] + n)
    s = {"case": case, "sizes": sizes, "tokens": tokens,
         "page_table": torch.tensor(table, **ints),
         "seq_lens": torch.tensor([l for _, l in sizes], **ints),
         "cu_tokens": torch.tensor(starts, **ints)}
    s["k_codes"], s["k_absmax"] = _filled(pages, case, gen, True)
    s["v_codes"], s["v_absmax"] = _filled(pages, case, gen, False)
    if case["rotary"]:
        half = case["rotary"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(case["longest"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    # one fused projection's output, of which queries, keys and values are slices
    if case["op"] != "read":
        h = case["heads"]
        fused = torch.empty((tokens, (h + 2 * hkv) * d), dtype=torch.float16, device="cuda")
        s["q"] = fused[:, :h * d].unflatten(1, (h, d))
        s["k"] = fused[:, h * d:(h + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = fused[:, (h + hkv) * d:].unflatten(1, (hkv, d))
        s["q"].copy_(torch.randn((tokens, h, d), device="cuda", generator=gen))
        s["k"].copy_(_values((tokens, hkv, d), gen, True))
        s["v"].copy_(_values((tokens, hkv, d), gen, False))
    if case["alibi"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["heads"] + 1, device="cuda")
                              / case["heads"])
    s["positions"] = torch.cat([torch.arange(l - n, l, device="cuda") for n, l in sizes])
    if case["op"] == "append":
        _plan_append(s, table)
    if own:
        _plan_own(s)
    return s


def _plan_append(s, table):
    """Index tensors a program would keep beside its page table: the blocks that
    hold new tokens, and where each of their tokens stands."""
    page = s["case"]["page"]
    block_page, block_slot, old, slot_of, out_of = [], [], [], [], []
    for b, (n, length) in enumerate(s["sizes"]):
        first = (length - n) // BLOCK
        for blk in range(first, -(-length // BLOCK)):
            for pos in range(blk * BLOCK, min(length, blk * BLOCK + BLOCK)):
                out_of.append(len(block_page) * BLOCK + pos - blk * BLOCK)
                if pos >= length - n:
                    slot_of.append(out_of[-1])
            old.append(max(0, length - n - blk * BLOCK))
            block_page.append(table[b][blk * BLOCK // page])
            block_slot.append(blk * BLOCK % page // BLOCK)
    s["block_page"] = torch.tensor(block_page, device="cuda")
    s["block_slot"] = torch.tensor(block_slot, device="cuda")
    s["block_old"] = torch.tensor(old, device="cuda")
    s["token_slot"] = torch.tensor(slot_of, device="cuda")
    s["out_slot"] = torch.tensor(out_of, device="cuda")


def _plan_own(s):
    from int8_quantized_matmul_absmax_amd import Int8KVCache, KVBatch, Rotary
    case = s["case"]
    s["cache"] = Int8KVCache.from_tensors(s["k_codes"], s["k_absmax"], s["v_codes"], s["v_absmax"])
    s["batch"] = KVBatch(s["page_table"], s["seq_lens"], s["cu_tokens"],
                         total_tokens=s["tokens"], max_tokens=max(n for n, _ in s["sizes"]),
                         max_len=max(l for _, l in s["sizes"]))
    s["rotary"] = Rotary(s["cos"], s["sin"], case["interleaved"]) if case["rotary"] else None
    if case["op"] == "append":
        # read back from the start of the first block that an append changes
        counts = [n + (l - n) % BLOCK for n, l in s["sizes"]]
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + c)
        s["changed"] = KVBatch(s["page_table"], s["seq_lens"],
                               torch.tensor(starts, dtype=torch.int32, device="cuda"),
                               total_tokens=starts[-1], max_tokens=max(counts),
                               max_len=max(l for _, l in s["sizes"]))


# --------------------------------------------------------------- plain forms

def _rotated(x, positions, s):
    """x [tokens, heads, dim] in 32 bits, its first `rotary` features rotated."""
    rot = s["case"]["rotary"]
    if not rot:
        return x
    cos, sin = s["cos"][positions][:, None], s["sin"][positions][:, None]
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _step(absmax):
    return absmax / torch.full_like(absmax, 127.0)


def _plain_append(s):
    outs = []
    hkv, d = s["case"]["kv_heads"], s["case"]["dim"]
    bp, bs = s["block_page"], s["block_slot"]
    row = torch.arange(BLOCK, device="cuda")
    is_old = row[None, :] < s["block_old"][:, None]
    for keys in (True, False):
        x = (s["k"] if keys else s["v"]).float()
        if keys:
            x = _rotated(x, s["positions"], s)
        codes, absmax = (s["k_codes"], s["k_absmax"]) if keys else (s["v_codes"], s["v_absmax"])
        new = torch.zeros((bp.numel() * BLOCK, hkv, d), device="cuda")
        new[s["token_slot"]] = x
        new = new.view(-1, BLOCK, hkv, d)
        was = torch.where(s["block_old"][:, None] > 0, absmax[bp, :, bs], 0.0)
        a = torch.maximum(was, new.abs().amax(dim=(1, 3)))
        safe = torch.where(a > 0, a, 1.0)
        old = codes[bp, :, bs].float()
        old = old.permute(0, 3, 1, 2, 4) if keys else old.permute(0, 4, 1, 2, 3)
        old = old.reshape(-1, BLOCK, hkv, d)
        kept = torch.round(old * (was / safe)[:, None, :, None])
        made = torch.round(new * (torch.full_like(safe, 127.0) / safe)[:, None, :, None])
        q = torch.where(is_old[:, :, None, None], kept, made)
        tiles = q.reshape(-1, BLOCK, hkv, d // 16, 16).to(torch.int8)
        tiles = tiles.permute(0, 2, 3, 1, 4) if keys else tiles.permute(0, 2, 3, 4, 1)
        codes[bp, :, bs] = tiles
        absmax[bp, :, bs] = a
        value = q * _step(a)[:, None, :, None]
        outs.append(value.reshape(-1, hkv, d)[s["out_slot"]].half())
    return tuple(outs)


def _cached(s, table, length):
    """Cached keys and values [rows, kv_heads, length, dim] in 32 bits."""
    outs = []
    table = table[:, :-(-length // s["case"]["page"])].clamp(min=0).long()
    for codes, absmax, order in ((s["k_codes"], s["k_absmax"], (0, 2, 1, 3, 5, 4, 6)),
                                 (s["v_codes"], s["v_absmax"], (0, 2, 1, 3, 6, 4, 5))):
        x = codes[table].float() * _step(absmax[table])[..., None, None, None]
        x = x.permute(order)   # [rows, heads, pages, slots, token, tile, feature]
        rows, heads = x.shape[:2]
        outs.append(x.reshape(rows, heads, -1, s["case"]["dim"])[:, :, :length])
    return outs


def _softmax_product(q, k, v, qpos, lengths, s):
    """q [rows, heads, n, dim], k and v [rows, kv_heads, length, dim]."""
    case = s["case"]
    rows, h, n, d = q.shape
    hkv, length = k.shape[1], k.shape[2]
    g = h // hkv
    z = torch.matmul(q.reshape(rows, hkv, g * n, d), k.transpose(2, 3).contiguous())
    z = z.view(rows, h, n, length) * (1.0 / math.sqrt(d))
    t = torch.arange(length, device="cuda")
    away = qpos[:, None, :, None] - t
    if case["alibi"]:
        z = z - s["slopes"][:, None, None] * away
    hidden = (away < 0) | (t >= lengths[:, None, None, None])
    if case["window"]:
        hidden = hidden | (away >= case["window"])
    z = z.masked_fill(hidden, -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(z - top)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(rows, hkv, g * n, length), v).view(rows, h, n, d)
    return o / torch.where(total > 0, total, 1.0)


def _plain_attention(s):
    case = s["case"]
    h, d = case["heads"], case["dim"]
    q = _rotated(s["q"].float(), s["positions"], s)
    out = torch.empty((s["tokens"], h, d), dtype=torch.float16, device="cuda")
    if case["new"] == 1:
        k, v = _cached(s, s["page_table"], case["longest"])
        o = _softmax_product(q[:, :, None], k, v, s["positions"][:, None], s["seq_lens"], s)
        out.copy_(o[:, :, 0])
        return out
    at = 0
    for b, (n, length) in enumerate(s["sizes"]):
        k, v = _cached(s, s["page_table"][b:b + 1], length)
        o = _softmax_product(q[None, at:at + n].transpose(1, 2), k, v,
                             s["positions"][None, at:at + n], s["seq_lens"][b:b + 1], s)
        out[at:at + n] = o[0].transpose(0, 1)
        at += n
    return out


def _plain_read(s):
    outs = ([], [])
    for b, (n, length) in enumerate(s["sizes"]):
        for out, x in zip(outs, _cached(s, s["page_table"][b:b + 1], length)):
            out.append(x[0, :, length - n:].transpose(0, 1).half())
    return tuple(torch.cat(out) for out in outs)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"attention": _plain_attention, "append": _plain_append,
                "read": _plain_read}[op](state)
    cache = state["cache"]
    if op == "attention":
        return cache.attention(state["q"], state["batch"], rotary=state["rotary"],
                               alibi_slopes=state.get("slopes"), window=state["case"]["window"])
    if op == "append":
        cache.append(state["k"], state["v"], state["batch"], rotary=state["rotary"])
        return cache.read(state["changed"])
    return cache.read(state["batch"])


# ------------------------------------------------------- definition, 64 bits

def _f64_rotation(x, positions, s):
    """Each pair of features as a complex number, times cos + i sin."""
    rot = s["case"]["rotary"]
    x = x.double()
    if not rot:
        return x
    turn = torch.complex(s["cos"].double()[positions], s["sin"].double()[positions])
    first = (slice(0, rot, 2), slice(1, rot, 2)) if s["case"]["interleaved"] else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., first[0]].contiguous(), x[..., first[1]].contiguous())
    z = z * turn[:, None, :]
    x[..., first[0]], x[..., first[1]] = z.real, z.imag
    return x


def _f64_token_codes(s, b, pos, keys):
    """Codes [tokens, heads, dim] and absmax [tokens, heads] of positions pos."""
    page = s["case"]["page"]
    p = s["page_table"][b].long()[torch.div(pos, page, rounding_mode="floor")]
    slot, t = pos % page // BLOCK, pos % BLOCK
    if keys:
        c = s["k_codes"][p, :, slot, :, t, :]
    else:
        c = s["v_codes"][p, :, slot, :, :, t]
    a = (s["k_absmax"] if keys else s["v_absmax"])[p, :, slot]
    return c.flatten(2).double(), a.double()


def _f64_values(s, b, pos, keys):
    c, a = _f64_token_codes(s, b, pos, keys)
    return c * a[..., None] / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "read":
        return tuple(torch.cat([_f64_values(s, b, torch.arange(l - n, l, device="cuda"), keys)
                                for b, (n, l) in enumerate(s["sizes"])]) for keys in (True, False))
    if case["op"] == "append":
        outs = []
        for keys in (True, False):
            x = s["k"] if keys else s["v"]
            x = _f64_rotation(x, s["positions"], s) if keys else x.double()
            rows, at = [], 0
            for b, (n, length) in enumerate(s["sizes"]):
                start = length - n
                edge = start // BLOCK * BLOCK
                pos = torch.arange(edge, length, device="cuda")
                new = x[at:at + n]
                at += n
                c, a = _f64_token_codes(s, b, pos[:start - edge], keys)
                blocks = torch.div(pos[start - edge:] - edge, BLOCK, rounding_mode="floor")
                top = torch.zeros((-(-(length - edge) // BLOCK), x.shape[1]),
                                  dtype=torch.float64, device="cuda")
                top.index_reduce_(0, blocks, new.abs().amax(dim=2), "amax")
                if start > edge:
                    top[0] = torch.maximum(top[0], a[0])
                top = top.clamp(min=1e-300)
                kept = torch.round(c * a[..., None] / top[0][:, None])
                made = torch.round(new * 127.0 / top[blocks][..., None])
                every = torch.div(pos - edge, BLOCK, rounding_mode="floor")
                rows.append(torch.cat((kept, made)) * top[every][..., None] / 127.0)
            outs.append(torch.cat(rows))
        return tuple(outs)
    q = _f64_rotation(s["q"], s["positions"], s)
    h, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((s["tokens"], h, d), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(s["sizes"]):
        pos = torch.arange(length, device="cuda")
        k, v = _f64_values(s, b, pos, True), _f64_values(s, b, pos, False)
        ahead = pos[None, :] - torch.arange(length - n, length, device="cuda")[:, None]
        seen = ahead <= 0
        if case["window"]:
            seen &= ahead > -case["window"]
        for j in range(h):
            i = j // (h // hkv)
            z = q[at:at + n, j] @ k[:, i].T / math.sqrt(d)
            if case["alibi"]:
                z = z + s["slopes"][j].double() * ahead
            p = torch.softmax(z.masked_fill(~seen, -math.inf), dim=-1)
            out[at:at + n, j] = p @ v[:, i]
        at += n
    return out
