"""What a serving loop decides between two model steps, on the GPU: Python binding of
include/batch.h.

    verify_drafts(target, draft_tokens, uniforms, cu_seqlens, *, draft_probs, temperature,
                  workspace) -> (tokens, num_accepted)
    batch_plan(lengths, rows, *, chunk_size, nchunks, context_lens, block_table, block_size)
                  -> BatchPlan

Checks are host checks of shapes, dtypes, strides and devices; kernels run on the current
stream (or `stream=`); nothing is copied to the host and nothing synchronises.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import library
from .attention import _run

__all__ = ["verify_drafts", "verify_workspace_bytes", "batch_plan", "BatchPlan"]


def verify_workspace_bytes(rows, nseq, vocab, scores=False):
    """Bytes a caller-provided `workspace` of verify_drafts must hold (scores: with
    temperature): the library's figure plus 255, since the binding aligns the start to 256."""
    return int(library().ssu_verify_workspace_bytes(rows, nseq, vocab, int(bool(scores)))) + 255


def verify_drafts(target, draft_tokens, uniforms, cu_seqlens, *, draft_probs=None,
                  temperature=None, workspace=None, stream=None):
    """Accepts or rejects drafted tokens and draws the next one. Returns (tokens, num_accepted),
    int32 [sequences, window + 1] and [sequences].

    Sequence b has n <= window drafts, draft_tokens[b, :n], and the 1 + n rows [cu_seqlens[b],
    cu_seqlens[b + 1]) of target [rows, vocab]: row i is the target's distribution p at the
    place of draft i, the last the one behind them. Draft i stands while uniforms[b, i] * q(x) <
    p(x), q being draft_probs[b, i] [vocab] or, without draft_probs, one at the draft. Behind the
    drafts that stand, a token is drawn with uniforms[b, window] from max(p - q, 0) (from p
    where no draft was rejected, or nothing is left): the lowest token at which the running sum
    passes uniforms[b, window] of the total. tokens[b] holds the accepted drafts and the
    drawn token, then -1; num_accepted[b] their number, which is what ssu_packed_varlen and
    linear_attention_packed take. Uniforms are fp32 in [0, 1).

    target holds probabilities, or with temperature (fp32 [sequences]) scores: p = softmax(score
    / temperature), and where the temperature is 0 or below, one at the largest score (the
    lowest token of equal ones). Probabilities p that are not above 0, NaN among them, and q below 0
    count as 0, NaN scores as minus infinity; a q of NaN rejects its draft and leaves its token out of
    the draw; a draft outside the vocabulary is rejected; where no token has any weight the drawn one
    is -1. A sequence without rows, with more than window
    + 1 or with rows outside the target gets tokens -1 and num_accepted 0."""
    return _run("verify", stream, target, draft_tokens, uniforms, cu_seqlens, draft_probs,
                temperature, workspace)


class BatchPlan(NamedTuple):
    """Tables of a packed batch, int32 on the GPU (row_slots int64)."""
    cu_seqlens: torch.Tensor                      # [requests + 1] first rows, then their number
    row_seq: torch.Tensor                         # [rows] request, -1 behind the last
    row_pos: torch.Tensor                         # [rows] position in it, -1 behind the last
    cu_chunk_seqlens: Optional[torch.Tensor]      # [nchunks + 1] first rows of chunks
    seq_idx: Optional[torch.Tensor]               # [nchunks] request of a chunk, -1 behind the last
    last_chunk_indices: Optional[torch.Tensor]    # [requests] last chunk, -1 if past nchunks
    row_slots: Optional[torch.Tensor]             # [rows] place in the blocks, -1 where none


def batch_plan(lengths, rows, *, chunk_size=None, nchunks=None, context_lens=None,
               block_table=None, block_size=1, stream=None):
    """Tables of `rows` packed rows that hold lengths[b] (int32 or int64, on the GPU) rows of
    each request, one request behind the other; rows behind the last stay without a request.
    In one launch and without the host knowing the lengths: a captured graph plans anew at
    every replay.

    row_pos counts from context_lens[b] (None: 0). With chunk_size, the tables of
    ssd_combined_fwd_varlen: every request is cut into chunks of at most chunk_size rows, one
    without rows has one empty chunk, which hands its state through; nchunks defaults to
    the most that there can be, rows // chunk_size + requests, and the chunks behind the last
    are empty and belong to no request. With block_table ([requests, blocks]), row_slots is
    block_table[b, row_pos // block_size] * block_size + row_pos % block_size: a row's
    place in a paged cache, or with block_size 1 in a table of state slots."""
    if chunk_size is None:
        if nchunks is not None:
            raise ValueError("nchunks needs a chunk_size")
    elif chunk_size < 1 or (nchunks is not None and nchunks < 0):
        raise ValueError("chunk_size must be positive and nchunks not negative")
    return BatchPlan(*_run("plan", stream, lengths, rows, chunk_size or 0,
                           -1 if nchunks is None else nchunks, context_lens, block_table,
                           block_size))
