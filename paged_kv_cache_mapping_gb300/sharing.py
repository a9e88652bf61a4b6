"""Binding of the entry points for requests that grow, shrink and share prompts
(include/pkv.h): the step's tables, the shared prefixes, and the attention that
reads each of them once.

Like the rest of the binding it only marshals arguments, through the compiled
module csrc/pkv_binding.cpp (the workspace's size through ctypes).
"""
import ctypes

import torch

from . import PkvError, _check, _tensor, speculative


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


def pkv_shared_attention_workspace_size(q, block_tables, k_cache, max_q_len: int = 0, max_group_len: int = 0) -> int:
    max_q_len, max_group_len = int(max_q_len), int(max_group_len)
    for name, x in (("max_q_len", max_q_len), ("max_group_len", max_group_len)):
        if x >= 1 << 31:  # ctypes would take its low 32 bits
            raise PkvError(1, f"{name} beyond int32")
    a = [_tensor(q, "q"), _tensor(block_tables, "block_tables"), _tensor(k_cache, "k_cache")]
    n = ctypes.c_size_t(0)
    _check(speculative._lib().pkv_shared_attention_workspace_size(*(ctypes.addressof(t) for t in a), max(max_q_len, 0),
                                                                  max(max_group_len, 0), ctypes.byref(n)))
    return int(n.value)


def pkv_shared_attention(q, cu_seqlens_q, seq_lens, block_tables, groups, k_cache, v_cache, scale: float, out,
                         k_scale: float = 1.0, v_scale: float = 1.0, max_q_len: int = 0, max_group_len: int = 0, workspace=None):
    """Causal attention of q [T, Hq, D] over the paged caches into out, where the requests of a group (groups [B, 3]: first
    request, request behind the last, tokens) read their common prefix once.  max_group_len bounds the rows of a group."""
    if workspace is None:
        workspace = torch.empty(pkv_shared_attention_workspace_size(q, block_tables, k_cache, max_q_len, max_group_len),
                                dtype=torch.uint8, device=q.device)
    rc = (speculative._calls or speculative._binding()).shared_attention(
        q, cu_seqlens_q, seq_lens, block_tables, groups, k_cache, v_cache, scale, k_scale, v_scale, max_q_len, max_group_len, out,
        workspace)
    if rc:
        _check(rc)
    return out
