"""The paged 8-bit key/value cache and what a call on it is given.

Int8KVCache holds the codes and absmaxes, KVBatch the sequences of a step and
Rotary the tables of a position rotation. Each checks its tensors once, when it
is made, so that the calls of a step's layers check only what is new to them.

    cache = Int8KVCache(num_pages, kv_heads, head_dim)        # one a layer
    batch = KVBatch(page_table, seq_lens, cu_tokens, ...)     # one a step
    cache.append(k, v, batch, rotary)
    y = cache.attention(q, batch, rotary)
"""

import collections
import ctypes

import torch

from . import _lib, ops
from .linear import shared_workspace

BLOCK = ops.KV_BLOCK
HEAD_DIMS = (64, 80, 96, 128, 256)


def _struct(cls, **fields):
    """A C struct and a reference to it (the object keeps both)."""
    s = cls(**fields)
    return s, ctypes.byref(s)


class Int8KVCache:
    """Keys and values as int8 codes with one absmax for each block of 16
    tokens and head, in pages of `page_tokens` tokens.

    k_codes, v_codes  int8 [num_pages, kv_heads, page_tokens / 16, D / 16, 16, 16]
                      tiles: keys [token][feature], values [feature][token]
    k_absmax, v_absmax  fp32 [num_pages, kv_heads, page_tokens / 16]
    k_means  None, or fp16 [num_pages, kv_heads, D]: the mean key of each page
             (page_means=True), which select_pages goes by

    Which page belongs to which sequence is the caller's to decide (KVPages)."""

    def __init__(self, num_pages, kv_heads, head_dim, page_tokens=64, device="cuda",
                 page_means=False):
        if head_dim not in HEAD_DIMS:
            raise ValueError("head_dim must be one of %s, got %s" % (HEAD_DIMS, head_dim))
        if page_tokens <= 0 or page_tokens % BLOCK != 0:
            raise ValueError("page_tokens must be a positive multiple of %d" % BLOCK)
        blocks = (int(num_pages), int(kv_heads), page_tokens // BLOCK)
        tiles = blocks + (head_dim // 16, 16, 16)
        self._hold(torch.empty(tiles, dtype=torch.int8, device=device),
                   torch.empty(blocks, dtype=torch.float32, device=device),
                   torch.empty(tiles, dtype=torch.int8, device=device),
                   torch.empty(blocks, dtype=torch.float32, device=device),
                   torch.zeros(blocks[:2] + (head_dim,), dtype=torch.float16, device=device)
                   if page_means else None)

    @classmethod
    def from_tensors(cls, k_codes, k_absmax, v_codes, v_absmax, k_means=None):
        """A cache over tensors of the layout above (shared, not copied)."""
        self = cls.__new__(cls)
        self._hold(k_codes, k_absmax, v_codes, v_absmax, k_means)
        return self

    def _hold(self, k_codes, k_absmax, v_codes, v_absmax, k_means=None):
        ops._need(k_codes, "k_codes", torch.int8, 6)
        pages, heads, slots, tiles = k_codes.shape[:4]
        if k_codes.shape[4:] != (16, 16) or tiles * 16 not in HEAD_DIMS or slots == 0 or heads == 0:
            raise ValueError("k_codes must be [pages, heads, blocks, D / 16, 16, 16] with D in %s, "
                             "got %s" % (HEAD_DIMS, tuple(k_codes.shape)))
        ops._need(k_absmax, "k_absmax", torch.float32, shape=(pages, heads, slots))
        ops._need(v_codes, "v_codes", torch.int8, shape=k_codes.shape)
        ops._need(v_absmax, "v_absmax", torch.float32, shape=(pages, heads, slots))
        if k_means is not None:
            ops._need(k_means, "k_means", torch.float16, shape=(pages, heads, tiles * 16))
        self.device = ops._on_gpu(k_codes=k_codes, k_absmax=k_absmax, v_codes=v_codes,
                                  v_absmax=v_absmax, k_means=k_means)
        self.k_codes, self.k_absmax = k_codes, k_absmax
        self.v_codes, self.v_absmax = v_codes, v_absmax
        self.k_means = k_means
        self.num_pages, self.kv_heads = pages, heads
        self.page_tokens, self.head_dim = slots * BLOCK, tiles * 16
        self._struct, self.ref = _struct(
            _lib.KVCacheStruct, k_codes=k_codes.data_ptr(), k_absmax=k_absmax.data_ptr(),
            v_codes=v_codes.data_ptr(), v_absmax=v_absmax.data_ptr(), num_pages=pages,
            page_tokens=self.page_tokens, kv_heads=heads, head_dim=self.head_dim)

    def append(self, k, v, batch, rotary=None):
        """Store the batch's new keys (rotated) and values; a cache that holds mean
        keys brings them up to date."""
        ops.int8_kv_cache_append(k, v, self, batch, rotary)
        if self.k_means is not None:
            ops.int8_kv_cache_page_means(self, batch)

    def attention(self, q, batch, rotary=None, scale=None, causal=True, window=0,
                  alibi_slopes=None, out=None):
        """Attention of the batch's queries over the cached tokens. Its workspace
        is the current stream's shared one (a graph's own while recording), as for
        the linear layers."""
        return ops.int8_kv_cache_attention(q, self, batch, rotary, scale, causal, window,
                                           alibi_slopes, shared_workspace, out)

    def update_means(self, batch):
        """The mean keys of the pages that hold the batch's tokens (append does this
        for its own; for keys that came into the cache another way)."""
        ops.int8_kv_cache_page_means(self, batch)

    def select_pages(self, q, batch, count, rotary=None, first=1, recent=1):
        """The pages that each new token and key/value head attends to, by its
        queries' products with the pages' mean keys: int32 [total_tokens, kv_heads,
        count]."""
        return ops.int8_kv_cache_select_pages(q, self, batch, count, rotary, first, recent)

    def attention_pages(self, q, pages, batch, rotary=None, scale=None, out=None):
        """Attention of the batch's queries over the tokens of the pages listed for
        each. Its workspace as for attention."""
        return ops.int8_kv_cache_attention_pages(q, pages, self, batch, rotary, scale,
                                                 shared_workspace, out)

    def read(self, batch):
        """Keys and values of the batch's tokens in fp16."""
        return ops.int8_kv_cache_read(self, batch)

    def copy_pages(self, copies):
        """The copies that a KVPages call asked for. The table it gave is right for
        this cache after them."""
        copies.pool.check(self)
        ops.int8_kv_cache_copy_pages(self, copies.pages, copies.counts)


class PageChoice(collections.namedtuple("PageChoice", "count first recent", defaults=(1, 1))):
    """How many pages a query attends to, and how many of them are always the first
    and the newest."""


class PageCopies:
    """Copies of pages that a KVPages call (of `pool`) asks for, on the GPU: pages int32
    [n, 3] (page, page to copy it to, tokens that count), counts int32 [2], the number
    of them first, and then, of a step, the pages that were wanting, of a compaction, the
    pages in use.

    Of a step also batch_lens int32 [rows], the lengths for a KVBatch of the new tokens,
    and full int32 [1], the rows that had no room for all of theirs (of a compaction
    None)."""

    def __init__(self, pages, counts, pool, step=None):
        self.pages, self.counts, self.pool, self._step = pages, counts, pool, step

    batch_lens = property(lambda self: self._step and self._step.batch_lens)
    full = property(lambda self: self._step and self._step.full)


class KVPages:
    """The pages of the caches of a model's layers, which share one page table. It
    holds nothing but their number and size: a page is free when no row of the table
    names it. Nothing waits for the host.

        table, lens, copies = pool.step(table, lens, parents)
        for cache in caches:
            cache.copy_pages(copies)
        batch = KVBatch(table, copies.batch_lens)"""

    def __init__(self, num_pages, page_tokens=64):
        if page_tokens <= 0 or page_tokens % BLOCK != 0:
            raise ValueError("page_tokens must be a positive multiple of %d" % BLOCK)
        if num_pages < 0:
            raise ValueError("num_pages must not be negative")
        self.num_pages, self.page_tokens = int(num_pages), int(page_tokens)

    def check(self, cache):
        """Refuses a cache that this pool's tables are not right for."""
        if cache.page_tokens != self.page_tokens or cache.num_pages < self.num_pages:
            raise ValueError("a cache of %d pages of %d tokens, the pool of %d of %d"
                             % (cache.num_pages, cache.page_tokens, self.num_pages,
                                self.page_tokens))

    def empty_table(self, rows, max_tokens, device="cuda"):
        """The table and lengths of `rows` sequences of no tokens, wide enough for
        max_tokens."""
        width = -(-int(max_tokens) // self.page_tokens)
        return (torch.full((rows, width), -1, dtype=torch.int32, device=device),
                torch.zeros((rows,), dtype=torch.int32, device=device))

    def step(self, page_table, seq_lens, parents, new_tokens=1, keep=None, max_len=None):
        """The table of the next step, its lengths (new tokens included) and the
        copies to make before its append. Row i keeps the first keep[i] tokens (None:
        all) of row parents[i] (-1: none) and has room for new_tokens (an int, or one
        a row) after them: beams that go on from others, prompts that several
        sequences share, growth, cutting back, beginning and, for rows that the new
        table leaves out, ending are all this call. Pages that rows share are copied
        for those about to write to them. copies.counts[1] says how many pages were
        wanting; their tokens are absent.

        The KVBatch of the new tokens takes copies.batch_lens: a row without new tokens
        has length 0 there, and so has one without room for all of them in the table (or
        below max_len, the batches'), whose tokens would be stored over its last ones, in
        pages that it may share. copies.full says how many those are; what the table
        holds of them stays."""
        step = ops._pages_step(page_table, seq_lens, parents, self.num_pages, self.page_tokens,
                               new_tokens, keep, shared_workspace, max_len)
        return step.table, step.lens, PageCopies(step.copies, step.counts, self, step)

    def compact(self, page_table, seq_lens):
        """The used pages to the front of the caches: the table with their new places
        and the copies to make. copies.counts[1] says how many are used."""
        table, pages, counts = ops.kv_pages_compact(page_table, seq_lens, self.num_pages,
                                                    self.page_tokens, shared_workspace)
        return table, PageCopies(pages, counts, self)


class KVBatch:
    """The sequences of one step (int32 tensors on the GPU; nothing waits for
    them on the host):

    page_table [num_seqs, max_pages], seq_lens [num_seqs] (new tokens included)
    cu_tokens  [num_seqs + 1] first row of each sequence's new tokens, the rows'
               total last; None: one new token a sequence
    total_tokens, max_tokens, max_len  the host's figures: rows of the packed
               tensors (default: num_seqs, without cu_tokens), and bounds on a
               sequence's new tokens (default: total_tokens) and on its length
               (default: what its row of the page table has room for). Rows that
               belong to no sequence get 0 from attention and read."""

    def __init__(self, page_table, seq_lens, cu_tokens=None, total_tokens=None, max_tokens=None,
                 max_len=None):
        ops._need(page_table, "page_table", torch.int32, 2)
        num_seqs = page_table.shape[0]
        ops._need(seq_lens, "seq_lens", torch.int32, shape=(num_seqs,))
        if cu_tokens is None:
            if total_tokens not in (None, num_seqs) or max_tokens not in (None, 1):
                raise ValueError("without cu_tokens each sequence has one new token")
            total_tokens, max_tokens = num_seqs, 1
        else:
            ops._need(cu_tokens, "cu_tokens", torch.int32, shape=(num_seqs + 1,))
            if total_tokens is None:
                raise ValueError("cu_tokens needs total_tokens")
            if max_tokens is None:
                max_tokens = total_tokens
        self.device = ops._on_gpu(page_table=page_table, seq_lens=seq_lens, cu_tokens=cu_tokens)
        self.page_table, self.seq_lens, self.cu_tokens = page_table, seq_lens, cu_tokens
        self.total_tokens, self.max_tokens = int(total_tokens), int(max_tokens)
        self.max_len = (1 << 30) if max_len is None else int(max_len)
        self._struct, self.ref = _struct(
            _lib.KVBatchStruct, page_table=page_table.data_ptr(), seq_lens=seq_lens.data_ptr(),
            cu_tokens=None if cu_tokens is None else cu_tokens.data_ptr(), num_seqs=num_seqs,
            max_pages=page_table.shape[1], total_tokens=self.total_tokens,
            max_tokens=self.max_tokens, max_len=self.max_len)


class Rotary:
    """Tables of a position rotation: cos, sin fp32 [positions, dim / 2]. Pairs
    are features (i, i + dim / 2), or (2 i, 2 i + 1) when interleaved."""

    def __init__(self, cos, sin, interleaved=False):
        ops._need(cos, "cos", torch.float32, 2)
        ops._need(sin, "sin", torch.float32, shape=cos.shape)
        self.device = ops._on_gpu(cos=cos, sin=sin)
        self.cos, self.sin, self.interleaved = cos, sin, bool(interleaved)
        self.positions, self.dim = cos.shape[0], 2 * cos.shape[1]
        self._struct, self.ref = _struct(
            _lib.RotaryStruct, cos=cos.data_ptr(), sin=sin.data_ptr(), dim=self.dim,
            positions=self.positions, interleaved=int(self.interleaved))
