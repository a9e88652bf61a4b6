"""Binding of the speculative decoding entry points (include/pkv.h): rotary
append, tree mask, tree attention and path commit.

Like the rest of the binding it only marshals arguments.  The calls that a
step makes once per layer, whose kernels take a few microseconds, go through
the compiled module csrc/pkv_binding.cpp; the others through ctypes.
"""
import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import PkvError, _check, _tensor, load_library

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "smooth": 4}


class Rope(ctypes.Structure):
    """The caller-kept pkv_rope: angles of a rotary embedding (pkv_rope_init)."""
    _fields_ = [("turns", ctypes.c_uint64 * 128), ("amplitude", ctypes.c_float), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("ready", ctypes.c_int32)]


class _RopeParams(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_max_position", ctypes.c_double), ("fast", ctypes.c_double), ("slow", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


_BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
_ready = None
_calls = None


def _lib():
    """The library with the argument types of these entry points."""
    global _ready
    if _ready is None:
        lib = load_library()
        p, f, i, z = ctypes.c_void_p, ctypes.c_float, ctypes.c_int32, ctypes.c_size_t
        for name, args in (("pkv_rope_init", [ctypes.POINTER(_RopeParams), ctypes.POINTER(Rope)]),
                           ("pkv_rope_append", [p, p, p, p, p, ctypes.POINTER(Rope), p, p, p, f, f, p]),
                           ("pkv_tree_mask", [p] * 6),
                           ("pkv_tree_attention_workspace_size", [p, p, p, i, ctypes.POINTER(z)]),
                           ("pkv_tree_attention", [p] * 7 + [f, f, f, i, p, p, z, p]),
                           ("pkv_tree_commit", [p] * 9)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _ready = lib
    return _ready


def _binding():
    """The compiled marshalling module, bound to the loaded library."""
    global _calls
    if _calls is None:
        lib = _lib()
        if not os.path.exists(_BINDING_PATH):
            raise PkvError(-1, f"{_BINDING_PATH} is missing: build it with "
                               "`python -m paged_kv_cache_mapping_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_binding", _BINDING_PATH)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
        loader.exec_module(m)
        at = lambda fn: ctypes.cast(fn, ctypes.c_void_p).value  # noqa: E731
        m.bind(PkvError, at(lib.pkv_rope_append), at(lib.pkv_tree_mask), at(lib.pkv_tree_attention), at(lib.pkv_tree_commit))
        _calls = m
    return _calls


def pkv_rope_init(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                  factor: float = 1.0, original_max_position: float = 0, fast: float = 0.0, slow: float = 0.0,
                  attention_factor: float = 0.0) -> Rope:
    """The angles of a rotary embedding, made once (host only) and passed to
    every pkv_rope_append.  scaling: "none", "linear", "ntk", "by_parts" or
    "smooth"; zeros take the defaults documented in include/pkv.h."""
    if scaling not in SCALINGS:
        raise PkvError(1, f"unknown scaling {scaling!r}: one of {', '.join(SCALINGS)}")
    a = _RopeParams(int(rot_dim), int(bool(interleaved)), SCALINGS[scaling], 0, float(base), float(factor),
                    float(original_max_position), float(fast), float(slow), float(attention_factor))
    rope = Rope()
    _check(_lib().pkv_rope_init(ctypes.byref(a), ctypes.byref(rope)))
    return rope


def pkv_rope_append(q, k, v, positions, slot_mapping, rope: Rope, k_cache, v_cache, q_out=None,
                    k_scale: float = 1.0, v_scale: float = 1.0):
    """Rotates q [T, Hq, D] and k [T, Hkv, D] by positions [T], writes k and v
    into their slots, and returns the rotated q (q_out, or a new tensor)."""
    if q_out is None:
        q_out = torch.empty_like(q)
    rc = (_calls or _binding()).rope_append(q, k, v, positions, slot_mapping, rope, q_out, k_cache, v_cache, k_scale, v_scale)
    if rc:
        _check(rc)
    return q_out


def pkv_tree_mask(parents, cu_seqlens_q, seq_lens, max_q_len: int, tree_mask=None, positions=None):
    """Mask words [T, ceil(max_q_len / 32)] and rotary positions [T] (int32) of
    drafted trees given as parent indices [T]."""
    rc, tree_mask, positions = (_calls or _binding()).tree_mask(parents, cu_seqlens_q, seq_lens, max_q_len, tree_mask,
                                                                positions)
    if rc:
        _check(rc)
    return tree_mask, positions


def pkv_tree_attention_workspace_size(q, block_tables, k_cache, max_q_len: int = 0) -> int:
    max_q_len = int(max_q_len)
    if max_q_len >= 1 << 31:  # ctypes would take its low 32 bits
        raise PkvError(1, "max_q_len beyond int32")
    a = [_tensor(q, "q"), _tensor(block_tables, "block_tables"), _tensor(k_cache, "k_cache")]
    n = ctypes.c_size_t(0)
    _check(_lib().pkv_tree_attention_workspace_size(*(ctypes.addressof(t) for t in a), max(max_q_len, 0), ctypes.byref(n)))
    return int(n.value)


def pkv_tree_attention(q, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, tree_mask, scale: float, out,
                       k_scale: float = 1.0, v_scale: float = 1.0, max_q_len: int = 0, workspace=None):
    """Attention of drafted trees q [T, Hq, D] over the paged caches into out:
    a node sees its sequence's context and the drafted nodes its mask names."""
    if workspace is None:
        workspace = torch.empty(pkv_tree_attention_workspace_size(q, block_tables, k_cache, max_q_len),
                                dtype=torch.uint8, device=q.device)
    rc = (_calls or _binding()).tree_attention(q, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, tree_mask, scale,
                                               k_scale, v_scale, max_q_len, out, workspace)
    if rc:
        _check(rc)
    return out


def pkv_tree_commit(accepted, accepted_lens, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache,
                    new_seq_lens=None):
    """Moves the accepted path's cache rows (accepted [B, A] node indices,
    accepted_lens [B]) to the front of the drafted rows, in place; returns the
    new lengths [B]."""
    if new_seq_lens is None:
        new_seq_lens = torch.empty_like(seq_lens)
    rc = (_calls or _binding()).tree_commit(accepted, accepted_lens, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache,
                                            new_seq_lens)
    if rc:
        _check(rc)
    return new_seq_lens
