"""Binding of the speculative decoding entry points (include/pkv.h): rotary
append, tree mask, tree attention and path commit.

Like the rest of the binding it only marshals arguments.  These calls are
made once per layer of a step whose kernels take a few microseconds, so the
tensors of a call are packed into one preallocated buffer per thread.
"""
import ctypes
import struct
import threading

import torch

from . import _DT, PkvError, _check, load_library

_TENSOR = struct.Struct("=Qii8q")  # pkv_tensor: data, dtype, ndim, shape[4], stride[4]
_PAD = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())
_MAX_TENSORS = 12
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


class _Buffer(threading.local):
    def __init__(self):
        self.buf = ctypes.create_string_buffer(_TENSOR.size * _MAX_TENSORS)
        at = ctypes.addressof(self.buf)
        self.at = [at + _TENSOR.size * i for i in range(_MAX_TENSORS)]


_buffer = _Buffer()
_ready = None


def _lib():
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


def _pack(*tensors):
    """Descriptors of (name, tensor) pairs, all on one CUDA device: that
    device's index and the addresses of the descriptors."""
    b = _buffer
    dev = -1
    for k, (name, t) in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        d = t.get_device()
        if d != dev or d < 0:
            if d < 0:
                raise PkvError(1, f"{name} must be a CUDA tensor (there is no CPU path)")
            if k:
                raise PkvError(1, f"{name} is on cuda:{d}, {tensors[0][0]} on cuda:{dev}")
            dev = d
        shape = t.shape
        n = len(shape)
        if n > 4:
            raise PkvError(1, f"{name} has more than 4 dimensions")
        dt = _DT.get(t.dtype)
        if dt is None:
            raise PkvError(2, f"{name}: unsupported dtype {t.dtype}")
        pad = _PAD[n]
        _TENSOR.pack_into(b.buf, k * _TENSOR.size, t.data_ptr(), dt, n, *shape, *pad, *t.stride(), *pad)
    return dev, b.at


def _call(dev, fn, *args):
    """fn(*args, stream) on dev's current stream, with dev current."""
    if torch.cuda.current_device() == dev:
        rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if rc:
        _check(rc)


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
    dev, a = _pack(("q", q), ("k", k), ("v", v), ("positions", positions), ("slot_mapping", slot_mapping),
                   ("q_out", q_out), ("k_cache", k_cache), ("v_cache", v_cache))
    _call(dev, _lib().pkv_rope_append, a[0], a[1], a[2], a[3], a[4], rope, a[5], a[6], a[7], k_scale, v_scale)
    return q_out


def pkv_tree_mask(parents, cu_seqlens_q, seq_lens, max_q_len: int, tree_mask=None, positions=None):
    """Mask words [T, ceil(max_q_len / 32)] and rotary positions [T] (int32) of
    drafted trees given as parent indices [T]."""
    if tree_mask is None:
        tree_mask = torch.empty((parents.shape[0], max(1, -(-int(max_q_len) // 32))), dtype=torch.int32,
                                device=parents.device)
    if positions is None:
        positions = torch.empty_like(parents)
    dev, a = _pack(("parents", parents), ("cu_seqlens_q", cu_seqlens_q), ("seq_lens", seq_lens),
                   ("tree_mask", tree_mask), ("positions", positions))
    _call(dev, _lib().pkv_tree_mask, a[0], a[1], a[2], a[3], a[4])
    return tree_mask, positions


def pkv_tree_attention_workspace_size(q, block_tables, k_cache, max_q_len: int = 0) -> int:
    _, a = _pack(("q", q), ("block_tables", block_tables), ("k_cache", k_cache))
    n = ctypes.c_size_t(0)
    _check(_lib().pkv_tree_attention_workspace_size(a[0], a[1], a[2], int(max_q_len), ctypes.byref(n)))
    return int(n.value)


def pkv_tree_attention(q, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, tree_mask, scale: float, out,
                       k_scale: float = 1.0, v_scale: float = 1.0, max_q_len: int = 0, workspace=None):
    """Attention of drafted trees q [T, Hq, D] over the paged caches into out:
    a node sees its sequence's context and the drafted nodes its mask names."""
    if workspace is None:
        workspace = torch.empty(pkv_tree_attention_workspace_size(q, block_tables, k_cache, max_q_len),
                                dtype=torch.uint8, device=q.device)
    dev, a = _pack(("q", q), ("cu_seqlens_q", cu_seqlens_q), ("seq_lens", seq_lens), ("block_tables", block_tables),
                   ("k_cache", k_cache), ("v_cache", v_cache), ("tree_mask", tree_mask), ("out", out))
    if workspace.get_device() != dev:
        raise PkvError(1, f"workspace must be on cuda:{dev}")
    _call(dev, _lib().pkv_tree_attention, a[0], a[1], a[2], a[3], a[4], a[5], a[6], scale, k_scale, v_scale,
          int(max_q_len), a[7], workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def pkv_tree_commit(accepted, accepted_lens, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache,
                    new_seq_lens=None):
    """Moves the accepted path's cache rows (accepted [B, A] node indices,
    accepted_lens [B]) to the front of the drafted rows, in place; returns the
    new lengths [B]."""
    if new_seq_lens is None:
        new_seq_lens = torch.empty_like(seq_lens)
    dev, a = _pack(("accepted", accepted), ("accepted_lens", accepted_lens), ("cu_seqlens_q", cu_seqlens_q),
                   ("seq_lens", seq_lens), ("block_tables", block_tables), ("k_cache", k_cache),
                   ("v_cache", v_cache), ("new_seq_lens", new_seq_lens))
    _call(dev, _lib().pkv_tree_commit, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7])
    return new_seq_lens
