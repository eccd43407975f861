"""Measured cases of generation over the paged 8-bit key/value cache: the choice
of a beam search's next beams, the step of the page tables that follows it with
the copies of shared pages, compaction, and attention over the pages that a
cheap score chooses for each query.

The cache holds int8 codes in 16 x 16 byte tiles, one absmax for each block of
16 tokens and head. Page p, head h, block s, tile c:
  k_codes[p, h, s, c, t, e]  key code of token 16 s + t, feature 16 c + e
  v_codes[p, h, s, c, e, t]  value code of the same token and feature
  k_absmax[p, h, s], v_absmax[p, h, s]; a code stands for code * absmax / 127.
k_means[p, h] is the mean of a page's keys in 16 bits.
"""

import math
import random

import torch

own = False

BLOCK = 16


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one search's next beams, with a small vocabulary: launch latency
        dict(name="beam_one", op="beam", batch=1, beams=4, vocab=32000, count=4, half=True),
        # a batch of searches, 32-bit logits, rows of an odd length, twice as many
        # candidates as beams, some beams ended, some searches at their first step
        dict(name="beam_16_odd", op="beam", batch=16, beams=5, vocab=50257, count=10, half=False),
        # a large serving batch over a large vocabulary: bandwidth
        dict(name="beam_64_wide", op="beam", batch=64, beams=8, vocab=131072, count=8, half=True),
        # one search of 4 beams early on, hidden size 4096 (32 heads of 128): latency
        dict(name="fork_one", op="fork", searches=1, beams=4, shortest=900, longest=1000,
             kv_heads=32, dim=128, page=64, spare=16, layers=1, new=1, cut=False),
        # 32 searches of 8 beams, grouped heads, every length, the pages of two layers
        dict(name="fork_32", op="fork", searches=32, beams=8, shortest=1, longest=8191,
             kv_heads=8, dim=128, page=64, spare=300, layers=2, new=1, cut=False),
        # a small pool after a few sequences have ended
        dict(name="compact_small", op="compact", rows=6, shortest=1, longest=1500, kv_heads=8,
             dim=64, page=48, ended=0.5, shared=0.0),
        # a serving pool of odd prompts, a third of it ended: bandwidth
        dict(name="compact_large", op="compact", rows=160, shortest=1, longest=8191, kv_heads=8,
             dim=128, page=64, ended=0.35, shared=0.25),
        # the pages for one token at the end of a very long document
        dict(name="select_one_long", op="select", batch=1, new=1, shortest=131071, longest=131071,
             heads=32, kv_heads=8, dim=128, page=128, rotary=128, interleaved=False, count=16,
             first=1, recent=2),
        # the pages for a serving batch, small pages
        dict(name="select_64", op="select", batch=64, new=1, shortest=100, longest=8192, heads=64,
             kv_heads=8, dim=128, page=16, rotary=64, interleaved=True, count=64, first=4,
             recent=8),
        # attention over them: one token of the long document
        dict(name="sparse_one_long", op="sparse", batch=1, new=1, shortest=131071, longest=131071,
             heads=32, kv_heads=8, dim=128, page=128, rotary=128, interleaved=False, count=16,
             first=1, recent=2),
        # the serving batch: cache bandwidth
        dict(name="sparse_64", op="sparse", batch=64, new=1, shortest=100, longest=8192, heads=64,
             kv_heads=8, dim=128, page=16, rotary=64, interleaved=True, count=64, first=4,
             recent=8),
        # ragged prompt chunks, each token with pages of its own: compute
        dict(name="sparse_chunks", op="sparse", batch=4, new=512, shortest=1, longest=16000,
             heads=32, kv_heads=8, dim=64, page=48, rotary=0, interleaved=False, count=32,
             first=1, recent=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("beam", "fork", "compact", "select", "sparse", "sparse"))
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        page = 16 * rng.randint(1, 8)
        dim = rng.choice((64, 80, 96, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 5, 8, 16, 32))
        if op == "beam":
            beams = rng.randint(1, 16)
            case = dict(batch=_log_int(rng, 1, 64), beams=beams, vocab=_log_int(rng, 500, 260000),
                        count=rng.choice((beams, 2 * beams, rng.randint(1, 32))),
                        half=rng.random() < 0.6)
        elif op == "fork":
            longest = _log_int(rng, 1, 16384)
            case = dict(searches=_log_int(rng, 1, 32), beams=rng.randint(1, 12),
                        shortest=rng.choice((1, longest)), longest=longest, kv_heads=kv_heads,
                        dim=dim, page=page, spare=_log_int(rng, 1, 500), layers=rng.randint(1, 2),
                        new=rng.choice((1, 1, rng.randint(0, 5), _log_int(rng, 1, 300))),
                        cut=rng.random() < 0.3)
        elif op == "compact":
            case = dict(rows=_log_int(rng, 1, 160), shortest=1, longest=_log_int(rng, 16, 8191),
                        kv_heads=kv_heads, dim=dim, page=page, ended=rng.uniform(0.1, 0.8),
                        shared=rng.choice((0.0, rng.random())))
        else:
            longest = _log_int(rng, 1, 131071)
            first, recent = rng.randint(0, 4), rng.randint(1, 8)
            case = dict(batch=_log_int(rng, 1, 64),
                        new=1 if rng.random() < 0.6 else _log_int(rng, 1, min(longest, 512)),
                        shortest=rng.choice((1, longest)), longest=longest,
                        heads=kv_heads * rng.choice((1, 1, 2, 3, 4, 6, 8)), kv_heads=kv_heads,
                        dim=dim, page=page, rotary=rng.choice((0, dim, dim // 32 * 16)),
                        interleaved=rng.random() < 0.3,
                        count=first + recent + _log_int(rng, 1, 120), first=first, recent=recent)
        case["op"] = op
        if _cost(case) <= most and _room(case) <= 3 << 29:
            return case


def _sizes(case):
    """(new tokens, length) of each sequence; the first is the longest."""
    rng = random.Random(case["longest"] * 101 + case.get("batch", 0) * 1000003 + case["page"])
    sizes = []
    for i in range(case["batch"]):
        n = case["new"] if i == 0 else rng.randint(1, case["new"])
        low = max(n, min(case["shortest"], case["longest"]))
        sizes.append((n, case["longest"] if i == 0 else rng.randint(low, case["longest"])))
    return sizes


def _page_bytes(case):
    blocks = case["page"] // BLOCK * case["kv_heads"]
    return blocks * (2 * BLOCK * case["dim"] + 8)


def _room(case):
    """Bytes that the case's caches (or, for beams, the plain form) hold at once."""
    if case["op"] == "beam":
        return 16 * case["batch"] * case["beams"] * case["vocab"]
    if case["op"] == "fork":
        plan = _fork_plan(case)
        return plan["pages"] * _page_bytes(case) * case["layers"]
    if case["op"] == "compact":
        return _compact_plan(case)["pages"] * _page_bytes(case)
    sizes = _sizes(case)
    cache = sum(-(-l // case["page"]) for _, l in sizes) * _page_bytes(case)
    # the plain form's scores of every page, and chosen pages of one sequence's tokens
    pages = -(-case["longest"] // case["page"])
    rows = case["batch"] if case["new"] == 1 else case["new"]
    if case["op"] == "select":
        return max(cache, 8 * rows * pages * case["kv_heads"] * case["dim"] // 4)
    return max(cache, 2 * rows * min(case["count"], pages) * case["page"] * case["dim"])


def work(case):
    op = case["op"]
    if op == "beam":
        rows = case["batch"] * case["beams"]
        return {"bytes": rows * case["vocab"] * (2 if case["half"] else 4)
                + 8 * rows + 16 * case["batch"] * case["count"],
                "flops": 4 * rows * case["vocab"]}
    if op == "fork":
        plan = _fork_plan(case)
        blocks = sum(-(-tokens // BLOCK) for _, _, tokens in _step(plan)[2])
        moved = blocks * case["kv_heads"] * (2 * BLOCK * case["dim"] + 8) * case["layers"]
        entries = sum(len(r) for r in plan["table"])
        return {"bytes": 2 * moved + 8 * entries, "flops": entries}
    if op == "compact":
        plan = _compact_plan(case)
        entries = sum(len(r) for r in plan["table"])
        return {"bytes": 2 * len(_compact(plan)[1]) * _page_bytes(case) + 8 * entries,
                "flops": entries}
    sizes = _sizes(case)
    d, hkv, h, page = case["dim"], case["kv_heads"], case["heads"], case["page"]
    tokens = sum(n for n, _ in sizes)
    table = 4 * case["rotary"] * tokens
    if op == "select":
        pages = sum(-(-l // page) for _, l in sizes)
        touched = sum((l - 1) // page - (l - n) // page + 1 for n, l in sizes)
        pairs = sum(-(-p // page) for n, l in sizes for p in range(l - n + 1, l + 1))
        return {"bytes": 2 * pages * hkv * d + touched * page * hkv * d + 2 * tokens * h * d + table
                + 4 * tokens * hkv * case["count"],
                "flops": 2 * d * hkv * pairs + 2 * touched * page * hkv * d}
    pairs, cached = 0, 0
    for n, l in sizes:
        seen = [min(p, case["count"] * page - (-p % page)) for p in range(l - n + 1, l + 1)]
        pairs += sum(seen)
        cached += min(l, sum(seen))
    return {"bytes": 2 * cached * hkv * d + 4 * tokens * h * d + table
            + 4 * tokens * hkv * case["count"],
            "flops": 4 * d * h * pairs}


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / 1e15


# ------------------------------------------------- page tables, on the host

def _fork_plan(case):
    """Searches whose beams share the pages of a prompt and have some of their own."""
    rng = random.Random(case["longest"] * 31 + case["searches"] * 1009 + case["beams"])
    page, beams = case["page"], case["beams"]
    table, lens, parents, new, keep, pages = [], [], [], [], [], 0
    for i in range(case["searches"]):
        length = case["longest"] if i == 0 else rng.randint(min(case["shortest"], case["longest"]),
                                                            case["longest"])
        prompt = (length - rng.randint(0, min(length, 600))) // page
        shared = list(range(pages, pages + prompt))
        pages += prompt
        for _ in range(beams):
            mine = -(-length // page) - prompt
            table.append(shared + list(range(pages, pages + mine)))
            pages += mine
            lens.append(length)
            parents.append(i * beams + min(int(rng.expovariate(0.5)), beams - 1))
            # a beam in ten has ended, a search in twenty is given up
            new.append(0 if rng.random() < 0.1 else case["new"])
            keep.append(length - rng.randint(0, min(length, 9)) if case["cut"] else length)
        if rng.random() < 0.05:
            parents[-beams:] = [-1] * beams
    pages += case["spare"]
    names = list(range(pages))
    rng.shuffle(names)
    room = -(-(max(lens) + case["new"]) // page) + 1
    return {"table": [[names[p] for p in r] for r in table], "lens": lens, "parents": parents,
            "new": new, "keep": keep, "pages": pages, "page": page, "room": room}


def _step(plan):
    """The definition of a step of the page tables: (table, lengths, copies, wanting)."""
    page, limit = plan["page"], plan["room"] * plan["page"]
    rows = []
    for parent, new, keep in zip(plan["parents"], plan["new"], plan["keep"]):
        old = parent if 0 <= parent < len(plan["lens"]) else None
        kept = 0 if old is None else min(keep, plan["lens"][old])
        length = min(kept + new, limit)
        mine = [] if old is None else plan["table"][old][:-(-kept // page)]
        rows.append((mine, kept, length, kept % page != 0 and length > kept))
    reading, first_writer = set(), {}
    for i, (mine, _, _, writes) in enumerate(rows):
        reading.update(mine[:-1] if writes else mine)
        if writes:
            first_writer.setdefault(mine[-1], i)
    used = set().union(*[r[0] for r in rows]) if rows else set()
    free = iter([p for p in range(plan["pages"]) if p not in used])
    table, lens, copies, wanting = [], [], [], 0
    for i, (mine, kept, length, writes) in enumerate(rows):
        mine = list(mine)
        if writes and (mine[-1] in reading or first_writer[mine[-1]] != i):
            source, mine[-1] = mine[-1], next(free, -1)
            if mine[-1] >= 0:
                copies.append((source, mine[-1], kept % page))
            wanting += mine[-1] < 0
        while len(mine) < -(-length // page):
            mine.append(next(free, -1))
            wanting += mine[-1] < 0
        table.append(mine)
        lens.append(length)
    return table, lens, copies, wanting


def _compact_plan(case):
    rng = random.Random(case["longest"] * 31 + case["rows"])
    page, table, lens, pages, before = case["page"], [], [], 0, []
    for i in range(case["rows"]):
        length = case["longest"] if i == 0 else rng.randint(case["shortest"], case["longest"])
        count = -(-length // page)
        # some begin with the pages of an earlier prompt
        shared = min(count - 1, len(before)) if rng.random() < case["shared"] else 0
        mine = before[:shared] + list(range(pages, pages + count - shared))
        pages += count - shared
        before = mine
        if i == 0 or rng.random() >= case["ended"]:
            table.append(mine)
            lens.append(length)
    pages += 5
    names = list(range(pages))
    rng.shuffle(names)
    return {"table": [[names[p] for p in r] for r in table], "lens": lens, "pages": pages,
            "page": page, "room": max(len(r) for r in table) + 1}


def _compact(plan):
    """The definition of a compaction: (table, copies, live pages)."""
    used = sorted({p for r in plan["table"] for p in r})
    live = len(used)
    there = set(used)
    to = dict(zip([p for p in used if p >= live], [p for p in range(live) if p not in there]))
    copies = [(a, b, plan["page"]) for a, b in to.items()]
    return [[to.get(p, p) for p in r] for r in plan["table"]], copies, live


def _padded(table, room):
    return torch.tensor([r + [-1] * (room - len(r)) for r in table], dtype=torch.int32,
                        device="cuda")


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
    codes = torch.empty((pages, hkv, slots, d // 16, 16, 16), dtype=torch.int8, device="cuda")
    absmax = torch.empty((pages, hkv, slots), device="cuda")
    step = max(1, (1 << 26) // (hkv * slots * BLOCK * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = _values((n, hkv, slots, BLOCK, d), gen, keys)
        a = x.abs().amax(dim=(3, 4))
        q = torch.round(x * (127.0 / a)[..., None, None]).to(torch.int8)
        q = q.view(n, hkv, slots, BLOCK, d // 16, 16)
        codes[at:at + n] = q.permute(0, 1, 2, 4, 3, 5) if keys else q.permute(0, 1, 2, 4, 5, 3)
        absmax[at:at + n] = a
    return codes, absmax


def _noise_cache(pages, case, gen):
    """A cache to be copied: what its codes are does not matter to a copy."""
    shape = (pages, case["kv_heads"], case["page"] // BLOCK)
    tiles = shape + (case["dim"] // 16, 16, 16)
    out = []
    for _ in range(2):
        out.append(torch.randint(-127, 128, tiles, dtype=torch.int8, device="cuda", generator=gen))
        out.append(torch.rand(shape, device="cuda", generator=gen) + 0.1)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = {"beam": _prepare_beam, "fork": _prepare_fork, "compact": _prepare_compact,
            "select": _prepare_pages, "sparse": _prepare_pages}[case["op"]]
    s = make(case, gen)
    s["case"] = case
    if own and case["op"] != "beam":
        from int8_quantized_matmul_absmax_amd import Int8KVCache, KVBatch, KVPages, Rotary
        if case["op"] in ("fork", "compact"):
            # (the caches' last page is a spare that the plain form writes to)
            s["pool"] = KVPages(s["pages"], case["page"])
            s["own_caches"] = [Int8KVCache.from_tensors(*c) for c in s["caches"]]
        else:
            s["cache"] = Int8KVCache.from_tensors(s["k_codes"], s["k_absmax"], s["v_codes"],
                                                  s["v_absmax"], k_means=s.get("k_means"))
            s["batch"] = KVBatch(s["page_table"], s["seq_lens"], s["cu_tokens"],
                                 total_tokens=s["tokens"],
                                 max_tokens=max(n for n, _ in s["sizes"]),
                                 max_len=case["longest"])
            s["rotary"] = Rotary(s["cos"], s["sin"], case["interleaved"]) if case["rotary"] \
                else None
    return s


def _prepare_beam(case, gen):
    b, k, v = case["batch"], case["beams"], case["vocab"]
    x = torch.randn((b, k, v), device="cuda", generator=gen) * 2.5
    # words that grammar or a stop list rules out
    x.masked_fill_(torch.rand((b, k, v), device="cuda", generator=gen) < 0.02, -math.inf)
    scores = -60.0 * torch.rand((b, k), device="cuda", generator=gen)
    scores = torch.sort(scores, dim=1, descending=True)[0].contiguous()
    first = torch.rand((b, 1), device="cuda", generator=gen) < 0.1
    scores = torch.where(first & (torch.arange(k, device="cuda") > 0), -math.inf, scores)
    live = torch.rand((b, k), device="cuda", generator=gen) >= 0.1
    live = (live | first).to(torch.int32)
    return {"logits": x.half() if case["half"] else x, "scores": scores, "live": live, "eos": 2}


def _prepare_fork(case, gen):
    plan = _fork_plan(case)
    ints = dict(dtype=torch.int32, device="cuda")
    return {"page_table": _padded(plan["table"], plan["room"]), "pages": plan["pages"],
            "seq_lens": torch.tensor(plan["lens"], **ints),
            "parents": torch.tensor(plan["parents"], **ints),
            "new": torch.tensor(plan["new"], **ints),
            "keep": torch.tensor(plan["keep"], **ints) if case["cut"] else None,
            "caches": [_noise_cache(plan["pages"] + 1, case, gen) for _ in range(case["layers"])]}


def _prepare_compact(case, gen):
    plan = _compact_plan(case)
    return {"page_table": _padded(plan["table"], plan["room"]), "pages": plan["pages"],
            "seq_lens": torch.tensor(plan["lens"], dtype=torch.int32, device="cuda"),
            "caches": [_noise_cache(plan["pages"] + 1, case, gen)]}


def _prepare_pages(case, gen):
    sizes, page, h = _sizes(case), case["page"], case["heads"]
    counts = [-(-l // page) for _, l in sizes]
    pages = sum(counts) + 2
    order = torch.randperm(pages, device="cuda", generator=gen).tolist()
    table, at = [], 0
    for c in counts:
        table.append(order[at:at + c])
        at += c
    ints = dict(dtype=torch.int32, device="cuda")
    starts = [0]
    for n, _ in sizes:
        starts.append(starts[-1] + n)
    tokens = starts[-1]
    s = {"sizes": sizes, "tokens": tokens, "page_table": _padded(table, max(counts)),
         "seq_lens": torch.tensor([l for _, l in sizes], **ints),
         "cu_tokens": torch.tensor(starts, **ints),
         "positions": torch.cat([torch.arange(l - n, l, device="cuda") for n, l in sizes])}
    s["k_codes"], s["k_absmax"] = _filled(pages, case, gen, True)
    if case["op"] == "select":
        s["v_codes"], s["v_absmax"] = s["k_codes"], s["k_absmax"]
        whole = torch.full((pages,), page, device="cuda")
        step = max(1, (1 << 26) // (page * case["kv_heads"] * case["dim"]))
        every = torch.arange(pages, device="cuda")
        s["case"] = case
        s["k_means"] = torch.cat([_plain_means(s, every[i:i + step], whole[i:i + step])
                                  for i in range(0, pages, step)])
        # what a program keeps beside its tables: the pages that hold new tokens
        touched = [(table[b][j], min(page, l - j * page)) for b, (n, l) in enumerate(sizes)
                   for j in range((l - n) // page, -(-l // page))]
        s["touched"] = torch.tensor([t[0] for t in touched], device="cuda")
        s["held"] = torch.tensor([t[1] for t in touched], device="cuda")
    else:
        s["v_codes"], s["v_absmax"] = _filled(pages, case, gen, False)
        s["chosen"] = _random_choice(case, s["positions"], gen)
    # queries are a slice of a fused projection's output
    fused = torch.empty((tokens, (h + 2 * case["kv_heads"]) * case["dim"]), dtype=torch.float16,
                        device="cuda")
    s["q"] = fused[:, :h * case["dim"]].unflatten(1, (h, case["dim"]))
    s["q"].copy_(torch.randn((tokens, h, case["dim"]), device="cuda", generator=gen))
    if case["rotary"]:
        half = case["rotary"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(case["longest"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    return s


def _random_choice(case, positions, gen):
    """Pages as a selection gives them: the first, the newest, others at random."""
    n, tokens, hkv = case["count"], positions.numel(), case["kv_heads"]
    out = torch.empty((tokens, hkv, n), dtype=torch.int32, device="cuda")
    pages = -(-case["longest"] // case["page"])
    step = max(1, (1 << 26) // (pages * hkv))
    for at in range(0, tokens, step):
        see = positions[at:at + step] // case["page"] + 1
        score = torch.rand((see.numel(), hkv, pages), dtype=torch.float64, device="cuda",
                           generator=gen)
        out[at:at + step] = _pick(score, see, case)
    return out


# --------------------------------------------------------------- plain forms

def _pick(score, see, case):
    """The pages of score [rows, heads, pages] for rows that see `see` pages."""
    n, pages = case["count"], score.shape[-1]
    j = torch.arange(pages, device="cuda")
    v = see[:, None, None]
    score = torch.where(torch.isnan(score), -math.inf, score)
    score = torch.where((j < case["first"]) | (j >= v - case["recent"]), math.inf, score)
    score = torch.where(j < v, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :n]
    best = torch.where(best < v, best, pages)
    best = torch.sort(best, dim=-1)[0]
    out = torch.full(score.shape[:2] + (n,), -1, dtype=torch.int32, device="cuda")
    out[..., :best.shape[-1]] = torch.where(best < pages, best, -1).to(torch.int32)
    return out


def _plain_beam(s):
    case = s["case"]
    b, k, v = s["logits"].shape
    n, kept = case["count"], min(case["count"], v)
    x = s["logits"].float() + 0.0          # (one zero)
    top = x.amax(dim=-1)
    alive = torch.isfinite(top)
    top = torch.where(alive, top, 0.0)
    total = torch.exp(x - top[..., None]).sum(dim=-1, dtype=torch.float64)
    base = s["scores"].double() - top.double() - torch.log(total)
    # values in order, the lower word first among equal ones
    bits = x.view(torch.int32)
    bits = bits ^ ((bits >> 31) & 0x7fffffff)
    keys = (bits.long() << 32) + ((1 << 32) - 1 - torch.arange(v, device="cuda"))
    best = torch.topk(keys, kept, dim=-1)[0]
    word = (1 << 32) - 1 - (best & ((1 << 32) - 1))
    value = base[..., None] + torch.gather(x, 2, word).double()
    value = torch.where(alive[..., None], value, -math.inf)
    # a beam that has ended goes on as it is
    ended = (s["live"] == 0)[..., None]
    at = torch.arange(kept, device="cuda")
    value = torch.where(ended, torch.where(at == 0, s["scores"].double()[..., None], -math.inf),
                        value)
    word = torch.where(ended, s["eos"], word)
    value, order = torch.sort(value.view(b, -1), dim=1, descending=True, stable=True)
    value, order = value[:, :n], order[:, :n]
    found = value > -math.inf
    word = torch.where(found, torch.gather(word.view(b, -1), 1, order), -1)
    parent = order // kept + torch.arange(b, device="cuda")[:, None] * k
    stay = torch.gather(s["live"], 1, order // kept) != 0
    parent = torch.where(found, parent, -1)
    live = found & stay & (word != s["eos"])
    outs = [value.float(), word.int(), parent.int(), live.int()]
    if value.shape[1] < n:
        fill = (-math.inf, -1, -1, 0)
        outs = [torch.cat((o, torch.full((b, n - o.shape[1]), f, dtype=o.dtype, device="cuda")), 1)
                for o, f in zip(outs, fill)]
    return tuple(outs)


def _plain_copies(s, copies):
    """Copies (source, target, tokens); rows of -1 write the spare page over itself."""
    spare = s["pages"]
    src = torch.where(copies[:, 0] < 0, spare, copies[:, 0]).long()
    dst = torch.where(copies[:, 1] < 0, spare, copies[:, 1]).long()
    slots = s["case"]["page"] // BLOCK
    moved = torch.arange(slots, device="cuda") * BLOCK < copies[:, 2:3]
    for cache in s["caches"]:
        for x in cache:
            m = moved.view((moved.shape[0], 1, slots) + (1,) * (x.dim() - 3))
            x[dst] = torch.where(m, x[src], x[dst])


def _plain_fork(s):
    table, page, pages = s["page_table"], s["case"]["page"], s["pages"]
    rows, room = s["parents"].numel(), table.shape[1]
    dev = dict(device="cuda")
    parent = s["parents"].long()
    valid = (parent >= 0) & (parent < table.shape[0])
    parent = parent.clamp(0, table.shape[0] - 1)
    held = torch.where(valid, s["seq_lens"][parent], 0)
    kept = held if s["keep"] is None else torch.minimum(s["keep"], held)
    length = (kept + s["new"]).clamp(max=room * page)
    kept_pages, all_pages = (kept + page - 1) // page, (length + page - 1) // page
    writes = (kept % page != 0) & (length > kept)
    j = torch.arange(room, **dev)
    inside = j < kept_pages[:, None]
    mine = torch.where(inside, table[parent], -1)
    last = (kept_pages - 1).clamp(min=0).long()
    partial = torch.gather(mine, 1, last[:, None])[:, 0]
    writes &= partial >= 0
    # pages kept by a row that will not write to them, and the first that will
    slot = torch.where(mine >= 0, mine, pages).long()
    reads = torch.where(writes[:, None] & (j == last[:, None]), pages, slot)
    reading = torch.zeros(pages + 1, dtype=torch.bool, **dev)
    reading[reads.view(-1)] = True
    used = torch.zeros(pages + 1, dtype=torch.bool, **dev)
    used[slot.view(-1)] = True
    row = torch.arange(rows, **dev)
    at = torch.where(writes, partial, pages).long()
    writer = torch.full((pages + 1,), rows, **dev).scatter_reduce(0, at, row, "amin")
    copy = writes & (reading[at] | (writer[at] != row))
    extra = all_pages - kept_pages
    need = copy.int() + extra
    begin = torch.cumsum(need, 0) - need
    free = torch.argsort(used[:pages].int(), stable=True)
    free_count = pages - used[:pages].sum()

    def take(n):
        return torch.where(n < free_count, free[n.clamp(max=pages - 1).long()], -1)

    dst = torch.where(copy, take(begin), partial)
    fresh = take(begin[:, None] + copy[:, None] + j - kept_pages[:, None])
    out = torch.where((j >= kept_pages[:, None]) & (j < all_pages[:, None]), fresh, mine)
    out = torch.where(copy[:, None] & (j == last[:, None]), dst[:, None], out).int()
    done = copy & (dst >= 0)
    place = torch.where(done, torch.cumsum(done, 0) - 1, rows)
    copies = torch.full((rows + 1, 3), -1, dtype=torch.int32, **dev)
    copies[place] = torch.stack((partial, dst, kept % page), 1).int()
    copies = copies[:rows]
    copies = torch.where((row < done.sum())[:, None], copies, -1)
    counts = torch.stack((done.sum(), (need.sum() - free_count).clamp(min=0))).int()
    _plain_copies(s, copies)
    return (out, length.int(), copies, counts) + tuple(x for c in s["caches"] for x in c)


def _plain_compact(s):
    table, page, pages = s["page_table"], s["case"]["page"], s["pages"]
    dev = dict(device="cuda")
    j = torch.arange(table.shape[1], **dev)
    inside = (j < ((s["seq_lens"] + page - 1) // page)[:, None]) & (table >= 0)
    slot = torch.where(inside, table, pages).long()
    used = torch.zeros(pages + 1, dtype=torch.bool, **dev)
    used[slot.view(-1)] = True
    used = used[:pages]
    live = used.sum()
    name = torch.arange(pages, **dev)
    moves, holes = used & (name >= live), ~used & (name < live)
    rank = torch.cumsum(moves, 0) - 1
    hole = torch.argsort((~holes).int(), stable=True)
    to = torch.where(moves, hole[rank.clamp(min=0)], name)
    out = torch.where(inside, to[slot.clamp(max=pages - 1)], -1).int()
    most = pages // 2
    copies = torch.full((most + 1, 3), -1, dtype=torch.int32, **dev)
    copies[torch.where(moves, rank, most)] = \
        torch.stack((name, to, torch.full_like(name, page)), 1).int()
    copies = torch.where((torch.arange(most, **dev) < moves.sum())[:, None], copies[:most], -1)
    counts = torch.stack((moves.sum(), live)).int()
    _plain_copies(s, copies)
    return (out, copies, counts) + tuple(x for c in s["caches"] for x in c)


def _step_of(absmax):
    return absmax / torch.full_like(absmax, 127.0)


def _plain_means(s, pages, held):
    """Means of the keys of `pages`, of which `held` tokens count."""
    case = s["case"]
    slots = case["page"] // BLOCK
    t = torch.arange(case["page"], device="cuda").view(slots, 1, BLOCK, 1)
    codes = torch.where(t < held.view(-1, 1, 1, 1, 1, 1), s["k_codes"][pages].double(), 0.0)
    sums = codes.sum(dim=4).flatten(3)     # [pages, heads, slots, dim]
    # a block past the end may hold anything, also a NaN
    step = torch.where(t[:, 0, 0, 0] < held.view(-1, 1, 1),
                       _step_of(s["k_absmax"][pages]).double(), 0.0)
    return ((sums * step[..., None]).sum(dim=2) / held.view(-1, 1, 1)).float().half()


def _turned(x, positions, s):
    """x [tokens, heads, dim] in its own type, its first `rotary` features rotated."""
    rot = s["case"]["rotary"]
    if not rot:
        return x
    cos, sin = (s[n][positions][:, None].to(x.dtype) for n in ("cos", "sin"))
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_select(s):
    case = s["case"]
    hkv, page = case["kv_heads"], case["page"]
    s["k_means"][s["touched"]] = _plain_means(s, s["touched"], s["held"])
    # in 64 bits: scores of two pages may be close to each other
    q = _turned(s["q"].double(), s["positions"], s)
    q = q.view(s["tokens"], hkv, -1, case["dim"]).sum(dim=2)
    see = s["positions"] // page + 1
    if case["new"] == 1:
        means = s["k_means"][s["page_table"].clamp(min=0).long()].double()
        score = torch.matmul(means.permute(0, 2, 1, 3), q[..., None])[..., 0]
        return s["k_means"], _pick(score, see, case)
    outs, at = [], 0
    for b, (n, length) in enumerate(s["sizes"]):
        means = s["k_means"][s["page_table"][b, :-(-length // page)].long()].double()
        score = torch.matmul(q[at:at + n].transpose(0, 1), means.permute(1, 2, 0).contiguous())
        outs.append(_pick(score.transpose(0, 1), see[at:at + n], case))
        at += n
    return s["k_means"], torch.cat(outs)


def _plain_sparse(s):
    case = s["case"]
    h, hkv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    g = h // hkv
    q = _turned(s["q"].float(), s["positions"], s).view(-1, hkv, g, d)
    seq = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"),
                                  s["cu_tokens"][1:] - s["cu_tokens"][:-1],
                                  output_size=s["tokens"])
    out = torch.empty((s["tokens"], hkv, g, d), dtype=torch.float16, device="cuda")
    offset = torch.arange(page, device="cuda")
    width = case["count"] * page
    step = max(1, (1 << 27) // (width * d))
    for i in range(hkv):
        for at in range(0, s["tokens"], step):
            j = s["chosen"][at:at + step, i].long()
            place = s["page_table"][seq[at:at + step, None], j.clamp(min=0)].long()
            x = s["k_codes"][place, i].float() * _step_of(s["k_absmax"][place, i])[..., None, None, None]
            k = x.permute(0, 1, 2, 4, 3, 5).reshape(-1, width, d)
            z = torch.matmul(q[at:at + step, i], k.transpose(1, 2).contiguous()) / math.sqrt(d)
            t = (j[..., None] * page + offset).view(-1, width)
            hidden = (j < 0)[..., None].expand(-1, -1, page).reshape(-1, width) \
                | (t > s["positions"][at:at + step, None])
            z = z.masked_fill(hidden[:, None], -math.inf)
            top = z.amax(dim=-1, keepdim=True)
            p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            total = p.sum(dim=-1, keepdim=True)
            x = s["v_codes"][place, i].float() * _step_of(s["v_absmax"][place, i])[..., None, None, None]
            v = x.permute(0, 1, 2, 5, 3, 4).reshape(-1, width, d)
            out[at:at + step, i] = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return out.view(-1, h, d)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"beam": _plain_beam, "fork": _plain_fork, "compact": _plain_compact,
                "select": _plain_select, "sparse": _plain_sparse}[op](s)
    if op == "beam":
        from int8_quantized_matmul_absmax_amd import beam_select
        return beam_select(s["logits"], s["scores"], s["live"], eos=s["eos"], count=case["count"])
    if op == "fork":
        table, lens, copies = s["pool"].step(s["page_table"], s["seq_lens"], s["parents"],
                                             new_tokens=s["new"], keep=s["keep"])
        for cache in s["own_caches"]:
            cache.copy_pages(copies)
        return (table, lens, copies.pages, copies.counts) + \
            tuple(x for c in s["caches"] for x in c)
    if op == "compact":
        table, copies = s["pool"].compact(s["page_table"], s["seq_lens"])
        for cache in s["own_caches"]:
            cache.copy_pages(copies)
        return (table, copies.pages, copies.counts) + tuple(x for c in s["caches"] for x in c)
    if op == "select":
        s["cache"].update_means(s["batch"])
        return s["k_means"], s["cache"].select_pages(s["q"], s["batch"], case["count"],
                                                     rotary=s["rotary"], first=case["first"],
                                                     recent=case["recent"])
    return s["cache"].attention_pages(s["q"], s["chosen"], s["batch"], rotary=s["rotary"])


# ------------------------------------------------------- definition, 64 bits

def _exact_beam(case, s):
    b, k, v = s["logits"].shape
    outs = []
    for i in range(b):
        value = torch.log_softmax(s["logits"][i].double(), dim=-1) + s["scores"][i].double()[:, None]
        for j in range(k):
            if not int(s["live"][i, j]):
                value[j] = -math.inf
                value[j, s["eos"]] = s["scores"][i, j].double()
        # (a row without words, all -infinity, has no softmax)
        value = torch.where(torch.isnan(value), -math.inf, value).view(-1)
        row = []
        for _ in range(case["count"]):
            best = float(value.max())
            if best == -math.inf:
                row.append((best, -1, -1, 0))
                continue
            at = int((value == best).nonzero()[0])
            value[at] = -math.inf
            row.append((best, at % v, i * k + at // v,
                        int(s["live"][i, at // v] != 0 and at % v != s["eos"])))
        outs.append(row)
    ints = dict(dtype=torch.int32, device="cuda")
    return (torch.tensor([[c[0] for c in r] for r in outs], dtype=torch.float64, device="cuda"),) + \
        tuple(torch.tensor([[c[n] for c in r] for r in outs], **ints) for n in (1, 2, 3))


def _exact_copied(case, s, copies, most, counts):
    """The list of copies, filled up with -1, and the caches after them."""
    for src, dst, tokens in copies:
        blocks = -(-tokens // BLOCK)
        for cache in s["caches"]:
            for x in cache:
                x[dst, :, :blocks] = x[src, :, :blocks]
    ints = dict(dtype=torch.int32, device="cuda")
    listed_copies = torch.tensor(copies + [(-1, -1, -1)] * (most - len(copies)), **ints)
    return (listed_copies.view(most, 3), torch.tensor(counts, **ints)) + \
        tuple(x for c in s["caches"] for x in c)


def _exact_keys(s, places, i, keys=True):
    """Tokens [rows, tokens, dim] of head i of pages [rows, n]."""
    codes, absmax = (s["k_codes"], s["k_absmax"]) if keys else (s["v_codes"], s["v_absmax"])
    rows = torch.arange(codes.shape[2], device="cuda")
    c = codes[places][:, :, i].double()
    if not keys:
        c = c.transpose(-1, -2)
    c = c * (absmax[places][:, :, i].double() / 127.0)[..., None, None, None]
    return c[:, :, rows].transpose(3, 4).flatten(4).flatten(1, 3)


def _exact_queries(s):
    """Each pair of features as a complex number, times cos + i sin."""
    rot, x = s["case"]["rotary"], s["q"].double()
    if not rot:
        return x
    turn = torch.complex(s["cos"].double()[s["positions"]], s["sin"].double()[s["positions"]])
    first = (slice(0, rot, 2), slice(1, rot, 2)) if s["case"]["interleaved"] else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., first[0]].contiguous(), x[..., first[1]].contiguous())
    z = z * turn[:, None, :]
    x[..., first[0]], x[..., first[1]] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    ints = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "beam":
        return _exact_beam(case, s)
    if case["op"] == "fork":
        plan = _fork_plan(case)
        table, lens, copies, wanting = _step(plan)
        return (_padded(table, plan["room"]), torch.tensor(lens, **ints)) + \
            _exact_copied(case, s, copies, len(lens), (len(copies), wanting))
    if case["op"] == "compact":
        plan = _compact_plan(case)
        table, copies, live = _compact(plan)
        return (_padded(table, plan["room"]),) + \
            _exact_copied(case, s, copies, plan["pages"] // 2, (len(copies), live))
    h, hkv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    q = _exact_queries(s)
    if case["op"] == "select":
        means = s["k_means"].double()
        for place, held in zip(s["touched"].tolist(), s["held"].tolist()):
            for i in range(hkv):
                # (a code stands for its product with the 32-bit quotient)
                step = (s["k_absmax"][place, i] / torch.full_like(s["k_absmax"][place, i], 127.0))
                c = s["k_codes"][place, i].double() * step.double()[:, None, None, None]
                means[place, i] = c.transpose(1, 2).flatten(2).flatten(0, 1)[:held].mean(dim=0)
        kept = means.float().half().double()   # as they are held
        rows, at = [], 0
        for b, (n, length) in enumerate(s["sizes"]):
            m = kept[s["page_table"][b, :-(-length // page)].long()]
            for r in range(at, at + n):
                p = int(length - n + r - at)
                v = p // page + 1
                score = torch.zeros((v, hkv), dtype=torch.float64, device="cuda")
                for j in range(h // hkv):
                    score += (m[:v] * q[r, j::h // hkv]).sum(dim=-1)
                score[:case["first"]] = math.inf
                score[max(0, v - case["recent"]):] = math.inf
                order = torch.sort(score, dim=0, descending=True, stable=True)[1][:case["count"]]
                line = torch.full((hkv, case["count"]), -1, **ints)
                line[:, :order.shape[0]] = torch.sort(order, dim=0)[0].T.int()
                rows.append(line)
            at += n
            if len(rows) > 3000:
                return None                     # (each row is sorted by itself)
        return means, torch.stack(rows)
    out = torch.zeros((s["tokens"], h, d), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // (case["count"] * page * d))
    at = 0
    for b, (n, length) in enumerate(s["sizes"]):
        for r in range(at, at + n, step):
            e = min(r + step, at + n)
            p = torch.arange(length - n + r - at, length - n + e - at, device="cuda")
            for i in range(hkv):
                j = s["chosen"][r:e, i].long()
                places = s["page_table"][b].long()[j.clamp(min=0)]
                t = j[:, :, None] * page + torch.arange(page, device="cuda")
                seen = ((j[:, :, None] >= 0) & (t <= p[:, None, None])).flatten(1)
                k, v = _exact_keys(s, places, i), _exact_keys(s, places, i, False)
                for c in range(i * (h // hkv), (i + 1) * (h // hkv)):
                    z = (k * q[r:e, c, None]).sum(dim=-1) / math.sqrt(d)
                    w = torch.softmax(z.masked_fill(~seen, -math.inf), dim=-1)
                    out[r:e, c] = (w[..., None] * v).sum(dim=1)
        at += n
    return out
