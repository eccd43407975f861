"""Int8CachedAttention: the attention layer of a decoder whose projections and
whose cache are int8.

A step takes the batch's new tokens through the fused query/key/value
projection (an Int8Linear), stores their keys and values in the layer's
Int8KVCache, attends over what the cache then holds, and takes the result
through the output projection. Prompt chunks, single tokens and mixtures of
both are one call: the KVBatch says which rows belong to which sequence. Over long
sequences a step may attend to some pages of the cache only (a PageChoice).

    attn = Int8CachedAttention(4096, 32, kv_heads=8)
    attn.quantize_(w_qkv, w_out)
    cache = Int8KVCache(num_pages, 8, 128)
    y = attn(x, cache, batch, rotary)          # x fp16 [total_tokens, 4096]
"""

import torch

from . import ops
from .linear import Int8Linear


class Int8CachedAttention(torch.nn.Module):
    """heads query heads share kv_heads (default: as many) key/value heads of
    head_dim (default hidden / heads) features. The rows of the fused weight are
    the query heads', then the key heads', then the value heads'."""

    def __init__(self, hidden, heads, kv_heads=None, head_dim=None, bias=False,
                 threshold=ops.DEFAULT_THRESHOLD, device="cuda"):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        if heads <= 0 or kv_heads <= 0 or heads % kv_heads != 0:
            raise ValueError("heads=%s is not a multiple of kv_heads=%s" % (heads, kv_heads))
        if head_dim is None:
            if hidden % heads != 0:
                raise ValueError("hidden=%s is not a multiple of heads=%s" % (hidden, heads))
            head_dim = hidden // heads
        self.hidden, self.heads, self.kv_heads = int(hidden), int(heads), int(kv_heads)
        self.head_dim = int(head_dim)
        self.qkv = Int8Linear(hidden, (heads + 2 * kv_heads) * head_dim, bias, threshold,
                              device=device)
        self.out = Int8Linear(heads * head_dim, hidden, bias, threshold, device=device)

    def quantize_(self, w_qkv, w_out, b_qkv=None, b_out=None):
        """Quantize the fp16 weights [(heads + 2 kv_heads) D, hidden] and
        [hidden, heads D] once."""
        self.qkv.quantize_(w_qkv, b_qkv)
        self.out.quantize_(w_out, b_out)
        return self

    def forward(self, x, cache, batch, rotary=None, scale=None, window=0, alibi_slopes=None,
                choice=None):
        """x fp16 [total_tokens, hidden], the batch's new tokens -> the same shape.
        choice (a PageChoice): each token attends to that many pages of its sequence,
        by a cache that holds mean keys, and not to all; without window and slopes."""
        if choice is not None and (window or alibi_slopes is not None):
            raise ValueError("a choice of pages has neither a window nor position biases")
        if choice is not None and cache.k_means is None:
            raise ValueError("the cache holds no mean keys (page_means=True)")
        if (cache.kv_heads, cache.head_dim) != (self.kv_heads, self.head_dim):
            raise ValueError("cache of %d heads of %d, layer of %d of %d"
                             % (cache.kv_heads, cache.head_dim, self.kv_heads, self.head_dim))
        if x.shape != (batch.total_tokens, self.hidden):
            raise ValueError("x must be [%d, %d], got %s"
                             % (batch.total_tokens, self.hidden, tuple(x.shape)))
        # heads of the projection's output as they lie: no copies
        y = self.qkv(x).view(batch.total_tokens, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = y.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        cache.append(k, v, batch, rotary)
        if choice is None:
            a = cache.attention(q, batch, rotary, scale=scale, window=window,
                                alibi_slopes=alibi_slopes)
        else:
            pages = cache.select_pages(q, batch, choice.count, rotary, choice.first, choice.recent)
            a = cache.attention_pages(q, pages, batch, rotary, scale=scale)
        return self.out(a.view(batch.total_tokens, self.heads * self.head_dim))
