"""Binding of the entry points for requests that grow, shrink and share prompts
(include/pkv.h): the step's tables and the shared prefixes.

Like the rest of the binding it only marshals arguments, through the compiled
module csrc/pkv_binding.cpp.
"""
import torch

from . import _check, speculative


def pkv_step_tables(seq_lens, new_seq_lens, block_tables, block_size: int, free_blocks, free_count, cu_seqlens_q, slot_mapping,
                    shared_blocks=None, positions=None, new_free_count=None):
    """Block tables [B, max_blocks] and the free list, updated in place for requests that go from seq_lens to new_seq_lens
    tokens [B]; writes cu_seqlens_q [B + 1], the new rows' slot_mapping [T] and positions [T], and the free blocks left
    (new_free_count [1], or free_count itself).  Returns cu_seqlens_q and slot_mapping."""
    rc = (speculative._calls or speculative._binding()).step_tables(
        seq_lens, new_seq_lens, shared_blocks, block_size, block_tables, free_blocks, free_count,
        free_count if new_free_count is None else new_free_count, cu_seqlens_q, slot_mapping, positions)
    if rc:
        _check(rc)
    return cu_seqlens_q, slot_mapping


def pkv_shared_prefixes(cu_seqlens_q, seq_lens, block_tables, block_size: int, min_tokens: int = 256, groups=None):
    """Groups [B, 3] (int32) of neighbouring requests whose tables begin with the same blocks: first request, request
    behind the last, tokens of their common prefix (0: alone)."""
    if groups is None:
        groups = torch.empty((seq_lens.shape[0], 3), dtype=torch.int32, device=seq_lens.device)
    rc = (speculative._calls or speculative._binding()).shared_prefixes(cu_seqlens_q, seq_lens, block_tables, block_size, min_tokens,
                                                                        groups)
    if rc:
        _check(rc)
    return groups
