"""Plain reference of the calls on page tables, in Python integers and sets, shared
with no GPU code. Tables are lists of rows of page numbers."""


def batch_lens(lens, parents, new, keep, limit):
    """-> (the rows' lengths in a batch of the new tokens: 0 where they have none or, of
    `limit` tokens, no room for all of them; how many have no room)."""
    out, full = [], 0
    for i, parent in enumerate(parents):
        k = min(max(lens[parent], 0), limit) if 0 <= parent < len(lens) else 0
        if keep is not None:
            k = min(k, max(keep[i], 0))
        fits = k + max(new[i], 0) <= limit
        out.append(k + new[i] if fits and new[i] > 0 else 0)
        full += not fits
    return out, full


def step(table, lens, parents, new, keep, num_pages, page, width, max_len=None):
    """-> (table of `width` entries a row, lengths, copies, wanting)."""
    limit = width * page if max_len is None else min(width * page, max_len)
    rows = []
    for i, parent in enumerate(parents):
        known = 0 <= parent < len(table)
        k = min(max(lens[parent], 0), limit) if known else 0
        if keep is not None:
            k = min(k, max(keep[i], 0))
        pages = [p if 0 <= p < num_pages else -1 for p in table[parent][:-(-k // page)]] \
            if known else []
        length = min(k + max(new[i], 0), limit)
        rows.append({"pages": pages, "kept": k, "len": length,
                     "writes": k % page != 0 and length > k})
    # who keeps each page without writing to it, and who will write
    readers, writers = {}, {}
    for i, r in enumerate(rows):
        for j, p in enumerate(r["pages"]):
            last = r["writes"] and j == len(r["pages"]) - 1
            (writers if last else readers).setdefault(p, []).append(i)
    kept = {p for r in rows for p in r["pages"]}
    free = [p for p in range(num_pages) if p not in kept]
    copies, wanting = [], 0

    def take():
        nonlocal wanting
        if free:
            return free.pop(0)
        wanting += 1
        return -1

    out, out_lens = [], []
    for i, r in enumerate(rows):
        pages = list(r["pages"])
        if r["writes"] and pages[-1] >= 0:
            p = pages[-1]
            if p in readers or writers[p][0] != i:
                pages[-1] = take()
                if pages[-1] >= 0:
                    copies.append((p, pages[-1], r["kept"] % page))
        while len(pages) < -(-r["len"] // page):
            pages.append(take())
        out.append(pages + [-1] * (width - len(pages)))
        out_lens.append(r["len"])
    return out, out_lens, copies, wanting


def compact(table, lens, num_pages, page):
    """-> (table, copies, used pages)."""
    rows = [[p if 0 <= p < num_pages else -1
             for p in r[:-(-min(max(l, 0), len(r) * page) // page)]] for r, l in zip(table, lens)]
    used = {p for r in rows for p in r if p >= 0}
    live = len(used)
    holes = [p for p in range(live) if p not in used]
    to = {p: p for p in used}
    copies = []
    for p in sorted(used):
        if p >= live:
            to[p] = holes.pop(0)
            copies.append((p, to[p], page))
    to[-1] = -1
    return [[to[p] for p in r] + [-1] * (len(t) - len(r)) for r, t in zip(rows, table)], copies, live


def copy(cache, copies, num_pages):
    """cache: dict of numpy arrays [pages, heads, slots, ...], changed in place."""
    for src, dst, tokens in copies:
        if not (0 <= src < num_pages and 0 <= dst < num_pages) or src == dst:
            continue
        for name, x in cache.items():
            if name == "k_means":
                if tokens > 0:
                    x[dst] = x[src]
            else:
                n = -(-max(tokens, 0) // 16)
                x[dst, :, :n] = x[src, :, :n]
