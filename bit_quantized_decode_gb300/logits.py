"""Penalties for repeated tokens, biases and grammar masks on rows of logits."""
from __future__ import annotations

import torch

from . import _lib


class LogitRules:
    """Rules of a batch of sequences over a vocabulary: ids int32 [S][cap], the tokens of each sequence, of which the first
    length[s] count and the first prompt[s] are its prompt (int32 [S]); repetition, frequency and presence float32 [S];
    bias_ids int32 and bias_values float32 [S][n].  The tensors stay on the device and may be updated in place between
    calls.  sequences: S, where nothing else says it."""

    def __init__(self, vocab: int, ids=None, length=None, prompt=None, repetition=None, frequency=None, presence=None,
                 bias_ids=None, bias_values=None, sequences: int = None):
        self.desc = _lib.logit_rules(vocab, ids, length, prompt, repetition, frequency, presence, bias_ids, bias_values, sequences)

    def __call__(self, logits, out=None, row_start=None, drafts=None, mask=None, allowed=None, flags: int = 0, stream=None):
        """The adjusted logits [R][V] of logits' type (out may be logits itself).  Row r is sequence r's, or sequence s has
        rows row_start[s] .. row_start[s + 1] - 1 (int32 [S + 1]): a drafted tree with tokens drafts (int32 [R]) and paths
        mask (int64 [R], bit j: the sequence's row j).  allowed: int32 [R][ceil(V / 32)], bit v % 32 of word v / 32."""
        if out is None:
            with _lib.allocating_on(stream):
                out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _lib.w4_logits_adjust(self.desc, logits, out, row_start, drafts, mask, allowed, flags, stream)
        return out
