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
"""
from __future__ import annotations

from typing import Optional


class DraftedBatch:
    """`seq_lens` (int32 [batch], kept and advanced in place): tokens cached for each of the first rows of `blocks`."""

    def __init__(self, blocks, seq_lens):
        from . import Places
        self.blocks, self.seq_lens = blocks, seq_lens
        self.places = Places(seq_lens.numel(), device=seq_lens.device)

    def begin(self, n_new: int, stream=None):
        """Blocks for n_new tokens of each sequence; returns how many got a place (int32 [batch], on the device)."""
        self.blocks.reserve(self.seq_lens, None, n_new, self.places, stream)
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
        """Verify the drafts against target [batch, drafts + 1, vocab]; the sequences keep the tokens that stand.
        Returns tq_verify_drafts' Verified: its last token of each sequence is the next step's first."""
        from . import _on, tq_verify_drafts
        verified = tq_verify_drafts(target, draft_tokens, draft_probs, uniforms, noise, temperatures, draft_lens, self.seq_lens,
                                    target_probs, out, stream)
        self.blocks.release(verified.keep_lens, stream)
        with _on(stream):
            self.seq_lens.copy_(verified.keep_lens)
        return verified
