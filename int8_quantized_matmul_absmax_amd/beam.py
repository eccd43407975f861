"""BeamSearch: a batch of beam searches over paged key/value caches.

Each search has `beams` rows of the page table. A step takes the logits of the rows'
last tokens, chooses the next beams, makes the next page table from the rows that
they go on from, and copies in every layer's cache the shared pages that two of them
are about to write to. Nothing waits for the host.

    table, lens, _ = pool.step(*pool.empty_table(searches, limit), none, new_tokens=prompt_lens)
    ...                                            # the prompts through the model
    search = BeamSearch(pool, caches, table, lens, beams=4, eos=2)
    tokens = search.step(logits)                   # [searches, 1, vocab] of the prompts' ends
    while ...:
        x = model(tokens.view(-1), caches, search.batch)
        tokens = search.step(x)                    # [searches, beams, vocab]
    tokens, scores = search.result()
"""

import torch

from . import ops
from .kv_cache import KVBatch
from .linear import shared_workspace


class BeamSearch:
    """pool and caches: the pages and the layers' caches that page_table (one row a
    search, its prompt's) is for. eos: the word that ends a beam, None if none does.
    max_len: a bound on the sequences' lengths for KVBatch (None: the table's width).

    page_table, seq_lens, scores, live: of the rows as they stand, ended beams
    included; batch: the KVBatch of the tokens that the last step chose; wanting: int32
    on the GPU, how many pages it found no room for (their tokens are absent); full:
    int32 on the GPU, how many beams had no room for their token in the table or below
    max_len. Such a beam keeps its tokens, but the new one is not stored and sees
    nothing: a search ends where full is not 0."""

    def __init__(self, pool, caches, page_table, seq_lens, beams, eos=None, max_len=None):
        searches = page_table.shape[0]
        if beams < 1 or beams > ops.MAX_BEAM_COUNT:
            raise ValueError("beams must be 1 .. %d, got %s" % (ops.MAX_BEAM_COUNT, beams))
        caches = list(caches)
        for c in caches:
            pool.check(c)
        self.pool, self.caches, self.beams, self.eos = pool, caches, int(beams), eos
        self.max_len = max_len
        self.page_table, self.seq_lens = page_table, seq_lens
        self.scores = torch.zeros((searches, 1), dtype=torch.float32, device=page_table.device)
        self.live = torch.ones((searches, 1), dtype=torch.int32, device=page_table.device)
        self.batch = self.wanting = self.full = None
        self._history = []

    def step(self, logits):
        """logits fp16 or fp32 [searches, rows, vocab], rows 1 in the first step and
        beams from then on -> the tokens int32 [searches, beams] to feed next (eos for
        a beam that has ended, -1 where there is none)."""
        self.scores, tokens, parents, self.live = ops.beam_select(
            logits, self.scores, self.live, self.eos, self.beams, shared_workspace)
        self.page_table, self.seq_lens, copies = self.pool.step(
            self.page_table, self.seq_lens, parents, new_tokens=self.live, max_len=self.max_len)
        for c in self.caches:
            c.copy_pages(copies)
        # (a beam that has ended, or is full, has length 0 there: it stores nothing)
        self.batch = KVBatch(self.page_table, copies.batch_lens, max_len=self.max_len)
        self.wanting, self.full = copies.counts[1], copies.full[0]
        self._history.append((tokens, parents))
        return tokens

    def result(self):
        """The beams' words so far, int32 [searches, beams, steps] (from its end on a
        beam repeats eos), and their scores, best first."""
        if not self._history:
            raise ValueError("no step has been taken")
        words = []
        at = torch.arange(self.scores.numel(), device=self.scores.device)
        there = torch.ones_like(at, dtype=torch.bool)
        for tokens, parents in reversed(self._history):
            words.append(torch.where(there, tokens.view(-1)[at], -1))
            up = parents.view(-1)[at]
            there = there & (up >= 0)
            at = up.clamp(min=0).long()
        words = torch.stack(words[::-1], dim=-1)
        return words.view(self.scores.shape + (len(self._history),)), self.scores
