"""The paged 8-bit key/value cache and what a call on it is given.

Int8KVCache holds the codes and absmaxes, KVBatch the sequences of a step and
Rotary the tables of a position rotation. Each checks its tensors once, when it
is made, so that the calls of a step's layers check only what is new to them.

    cache = Int8KVCache(num_pages, kv_heads, head_dim)        # one a layer
    batch = KVBatch(page_table, seq_lens, cu_tokens, ...)     # one a step
    cache.append(k, v, batch, rotary)
    y = cache.attention(q, batch, rotary)
"""

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

    Which page belongs to which sequence is the caller's to decide."""

    def __init__(self, num_pages, kv_heads, head_dim, page_tokens=64, device="cuda"):
        if head_dim not in HEAD_DIMS:
            raise ValueError("head_dim must be one of %s, got %s" % (HEAD_DIMS, head_dim))
        if page_tokens <= 0 or page_tokens % BLOCK != 0:
            raise ValueError("page_tokens must be a positive multiple of %d" % BLOCK)
        blocks = (int(num_pages), int(kv_heads), page_tokens // BLOCK)
        tiles = blocks + (head_dim // 16, 16, 16)
        self._hold(torch.empty(tiles, dtype=torch.int8, device=device),
                   torch.empty(blocks, dtype=torch.float32, device=device),
                   torch.empty(tiles, dtype=torch.int8, device=device),
                   torch.empty(blocks, dtype=torch.float32, device=device))

    @classmethod
    def from_tensors(cls, k_codes, k_absmax, v_codes, v_absmax):
        """A cache over tensors of the layout above (shared, not copied)."""
        self = cls.__new__(cls)
        self._hold(k_codes, k_absmax, v_codes, v_absmax)
        return self

    def _hold(self, k_codes, k_absmax, v_codes, v_absmax):
        ops._need(k_codes, "k_codes", torch.int8, 6)
        pages, heads, slots, tiles = k_codes.shape[:4]
        if k_codes.shape[4:] != (16, 16) or tiles * 16 not in HEAD_DIMS or slots == 0 or heads == 0:
            raise ValueError("k_codes must be [pages, heads, blocks, D / 16, 16, 16] with D in %s, "
                             "got %s" % (HEAD_DIMS, tuple(k_codes.shape)))
        ops._need(k_absmax, "k_absmax", torch.float32, shape=(pages, heads, slots))
        ops._need(v_codes, "v_codes", torch.int8, shape=k_codes.shape)
        ops._need(v_absmax, "v_absmax", torch.float32, shape=(pages, heads, slots))
        self.device = ops._on_gpu(k_codes=k_codes, k_absmax=k_absmax, v_codes=v_codes,
                                  v_absmax=v_absmax)
        self.k_codes, self.k_absmax = k_codes, k_absmax
        self.v_codes, self.v_absmax = v_codes, v_absmax
        self.num_pages, self.kv_heads = pages, heads
        self.page_tokens, self.head_dim = slots * BLOCK, tiles * 16
        self._struct, self.ref = _struct(
            _lib.KVCacheStruct, k_codes=k_codes.data_ptr(), k_absmax=k_absmax.data_ptr(),
            v_codes=v_codes.data_ptr(), v_absmax=v_absmax.data_ptr(), num_pages=pages,
            page_tokens=self.page_tokens, kv_heads=heads, head_dim=self.head_dim)

    def append(self, k, v, batch, rotary=None):
        """Store the batch's new keys (rotated) and values."""
        ops.int8_kv_cache_append(k, v, self, batch, rotary)

    def attention(self, q, batch, rotary=None, scale=None, causal=True, window=0,
                  alibi_slopes=None, out=None):
        """Attention of the batch's queries over the cached tokens. Its workspace
        is the current stream's shared one (a graph's own while recording), as for
        the linear layers."""
        return ops.int8_kv_cache_attention(q, self, batch, rotary, scale, causal, window,
                                           alibi_slopes, shared_workspace, out)

    def read(self, batch):
        """Keys and values of the batch's tokens in fp16."""
        return ops.int8_kv_cache_read(self, batch)


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
