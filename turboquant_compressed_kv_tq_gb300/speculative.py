"""A batch of sequences that grows by drafted tokens, over a block table.

A speculative step ("lightning-mlx/plan.md": several tokens verified at one read of
the cache) runs each sequence's newest token and the drafts behind it through the
model at once. Around the model's layers it is

  1. ``begin``: blocks for the step's tokens (``tq_blocks_reserve``);
  2. in each layer ``rotate`` (``tq_rope_apply`` at the tokens' positions) and
     ``attend`` (``tq_decode_step``: append them, attend over the grown sequences);
  3. ``finish``: which drafts stand and the token behind them
     (``tq_verify_drafts``), and the blocks behind them back (``tq_blocks_release``).

All lengths stay on the device, so that the steps can be captured into a CUDA graph;
this module holds the order of the calls, the arithmetic runs in the library's kernels.

Where the free list or a sequence's row of the table has not blocks for all tokens of a
step, the sequence stands still: it keeps its length, gives back what it got, and its
tokens are -1 (TQ_DEVERR_CAPACITY tells, and the attention sets TQ_DEVERR_BLOCK or
TQ_DEVERR_SEQLEN). A part of the tokens would not do: the decode kernels leave
out tiles of up to 64 tokens in which a block is missing, so that what the others attended to is
not known. The same step again goes on as soon as there are blocks; a row that is nearly full
takes shorter steps. Every sequence takes part in every step: one that has ended is taken
out of the batch by the caller (``tq_batch_filter``), or its row is begun anew.
"""
from __future__ import annotations

from typing import Optional


class DraftedBatch:
    """`seq_lens` (int32 [batch], kept and advanced in place): tokens cached for each of the first rows of `blocks`."""

    def __init__(self, blocks, seq_lens):
        import torch
        from . import Places
        self.blocks, self.seq_lens = blocks, seq_lens
        self.places = Places(seq_lens.numel(), device=seq_lens.device)
        self.n_new = None   # of the step that has begun
        # sequences that have not a place for each of its tokens
        self._short = torch.zeros_like(seq_lens, dtype=torch.bool)
        self._short_rows = self._short[:, None]

    def begin(self, n_new: int, stream=None):
        """Blocks for n_new tokens of each sequence; returns how many got a place (int32 [batch], on the device). A sequence
        with fewer than n_new takes no part in the step."""
        self.blocks.reserve(self.seq_lens, None, n_new, self.places, stream)
        self.n_new = n_new
        return self.places.granted

    def rotate(self, rope, q, k, out=None, k_out=None, stream=None):
        """q and k [batch, heads, n_new, head_dim] at the step's positions: contiguous, as `attend` takes them."""
        return rope.apply(q, k, out, k_out, starts=self.seq_lens, stream=stream)

    def attend(self, cache, layer, k, v, q, max_seq_len, out, workspace, scale=0.0, stream=None):
        """Append the step's keys and values to a layer and attend with its queries."""
        cache.decode_step(layer, k, v, q, self.seq_lens, self.blocks.table, self.blocks.max_blocks, max_seq_len, out,
                          workspace, scale, stream)

    def finish(self, target, draft_tokens=None, draft_probs=None, uniforms=None, noise=None, temperatures=None,
               draft_lens=None, target_probs=False, out: Optional[object] = None, stream=None):
        """Verify the drafts against target [batch, drafts + 1, vocab], drafts + 1 at most the step's tokens; the sequences keep
        the tokens that stand. Returns tq_verify_drafts' Verified: its last token of each sequence is the next step's first
        (tokens of -1: the sequence stood still, and its first token is the one that it had)."""
        from . import _here, _on, tq_verify_drafts
        if self.n_new is not None and target.dim() == 3 and target.shape[1] > self.n_new:
            raise ValueError(f"target has {target.shape[1]} rows a sequence, the step {self.n_new} tokens")
        with _on(stream) if stream is not None else _here:
            before = self.seq_lens
            if out is not None and out.keep_lens is not None and out.keep_lens.data_ptr() == before.data_ptr():   # (in place)
                before = before.clone()
            verified = tq_verify_drafts(target, draft_tokens, draft_probs, uniforms, noise, temperatures, draft_lens, self.seq_lens,
                                        target_probs, out, stream)
            if self.n_new is not None:
                self._stand_still(verified, before)
            self.blocks.release(verified.keep_lens, stream)
            self.seq_lens.copy_(verified.keep_lens)   # (what is returned stays as it is in the next step)
        return verified

    def _stand_still(self, verified, before):
        import torch
        torch.ne(self.places.granted, self.n_new, out=self._short)
        torch.where(self._short, before, verified.keep_lens, out=verified.keep_lens)
        verified.accepted.masked_fill_(self._short, 0)
        verified.tokens.masked_fill_(self._short_rows, -1)
        if verified.logprobs is not None:
            verified.logprobs.masked_fill_(self._short_rows, 0.0)
