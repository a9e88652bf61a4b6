"""Outputs of the speculative calls that overlap what the call reads are
refused on the host (no GPU): CTAs that are still reading would see them."""
import ctypes
import random

import pytest
import torch

from paged_kv_cache_mapping_gb300 import build as pkv_build
from paged_kv_cache_mapping_gb300 import speculative as spec
from tests.test_abi import BF16, FAKE, I32, _t

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return spec._lib()


def ptr(x):
    return ctypes.addressof(x)


# ---------------------------------------------------------------- commit
AT = {"acc": 0x100000, "lens": 0x200000, "cu": 0x300000, "sl": 0x400000, "bt": 0x500000, "kc": 0x600000, "vc": 0x700000}


@pytest.mark.parametrize("over,by", [("sl", 0), ("lens", 0), ("lens", 4), ("lens", -4), ("cu", 8), ("acc", 16), ("acc", 28), ("bt", 0),
                                     ("kc", 64), ("vc", 0)])
def test_new_lengths_of_a_commit(lib, over, by):
    a = dict(acc=_t(FAKE + AT["acc"], I32, [2, 4]), lens=_t(FAKE + AT["lens"], I32, [2]), cu=_t(FAKE + AT["cu"], I32, [3]),
             sl=_t(FAKE + AT["sl"], I32, [2]), bt=_t(FAKE + AT["bt"], I32, [2, 5]), kc=_t(FAKE + AT["kc"], BF16, [10, 16, 2, 64]),
             vc=_t(FAKE + AT["vc"], BF16, [10, 16, 2, 64]), new=_t(FAKE + AT[over] + by, I32, [2]))
    assert lib.pkv_tree_commit(*(ptr(a[k]) for k in ("acc", "lens", "cu", "sl", "bt", "kc", "vc", "new")), None) == INVALID
    assert b"new_seq_lens must not overlap" in lib.pkv_last_error()


# ---------------------------------------------------------------- rotary append
PASSED = 4  # no GPU here: the first CUDA call after the checks fails
Q0 = FAKE + 0x100000


def fused(part, T=6, Hq=8, Hkv=2, D=64, at=Q0):
    """A part of [T, Hq + 2 Hkv, D] rows."""
    h0, h = {"q": (0, Hq), "k": (Hq, Hkv), "v": (Hq + Hkv, Hkv)}[part]
    return _t(at + h0 * D * 2, BF16, [T, h, D], [(Hq + 2 * Hkv) * D, D, 1])


def plain(at, T=6, H=8, D=64, st=None, sh=64):
    return _t(at, BF16, [T, H, D], [H * D if st is None else st, sh, 1])


far = FAKE + 0x10000000
CASES = {
    "fused, in place": (fused("q"), fused("k"), fused("v"), fused("q"), True),
    "fused, elsewhere": (fused("q"), fused("k"), fused("v"), plain(far), True),
    "over k": (fused("q"), fused("k"), fused("v"), fused("q", at=Q0 + 8 * 64 * 2), False),
    "over v by a head": (fused("q"), fused("k"), fused("v"), fused("q", at=Q0 - 64 * 2 * 3 + 12 * 64 * 2), False),
    "one row on": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0 + 128), False),
    "one token on": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0 + 8 * 128), False),
    "half a row back": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0 - 64), False),
    "the last row": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0 + 6 * 8 * 128 - 128), False),
    "behind": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0 + 6 * 8 * 128), True),
    "before": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0 - 6 * 8 * 128), True),
    "tokens in turn": (plain(Q0, st=1024), plain(far, H=2), plain(far, H=2), plain(Q0 + 1024, st=1024), True),
    "tokens in turn, too near": (plain(Q0, st=1024), plain(far, H=2), plain(far, H=2), plain(Q0 + 1008, st=1024), False),
    "heads in turn": (plain(Q0, st=1024, sh=128), plain(far, H=2), plain(far, H=2), plain(Q0 + 128, st=1024, sh=128), True),
    "other strides": (plain(Q0), plain(far, H=2), plain(far, H=2), plain(Q0, st=1024), False),
    "one token, other strides": (plain(Q0, T=1), plain(far, T=1, H=2), plain(far, T=1, H=2), plain(Q0, T=1, st=1024), True),
    "one token, one row on": (plain(Q0, T=1), plain(far, T=1, H=2), plain(far, T=1, H=2), plain(Q0 + 128, T=1), False),
    "no token": (plain(Q0, T=0), plain(far, T=0, H=2), plain(far, T=0, H=2), plain(Q0 + 128, T=0), True),
}


def append(lib, q, k, v, o, kc, T, rot):
    if torch.cuda.is_available():
        pytest.skip("what passes the checks would be launched")
    index = _t(FAKE, I32, [T])
    return lib.pkv_rope_append(ptr(q), ptr(k), ptr(v), ptr(index), ptr(index), spec.pkv_rope_init(rot), ptr(o), ptr(kc), ptr(kc), 1.0,
                               1.0, None)


@pytest.mark.parametrize("name", list(CASES))
def test_rotated_rows(lib, name):
    q, k, v, o, fine = CASES[name]
    T, kc = q.shape[0], _t(FAKE, BF16, [10, 16, 2, 64])
    rc = append(lib, q, k, v, o, kc, T, 64)
    assert rc == (PASSED if fine else INVALID), lib.pkv_last_error()
    if not fine:
        assert b"overlap" in lib.pkv_last_error()


def test_rows_overlap_by_brute_force(lib):
    """The host's rule against every byte of every row, for views of one buffer."""
    r = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        T, H, J, D = r.randint(1, 4), r.randint(1, 4), r.randint(1, 4), 8
        sh = r.choice([D, 2 * D, 3 * D])
        st = r.choice([sh * max(H, J), sh * max(H, J) + D, sh * (H + J), 40 * D, D])
        if st == D:  # tokens inside, heads outside
            st, sh = r.choice([D, 2 * D]), 16 * D
        d = 8 * r.randint(-20 * D // 8, 40 * D // 8)
        q = _t(far, BF16, [T, H, D], [st, sh, 1])
        k, o = _t(Q0, BF16, [T, J, D], [st, sh, 1]), _t(Q0 + 2 * d, BF16, [T, H, D], [st, sh, 1])
        byte = lambda x, n: {x.data + 2 * (t * st + h * sh) + e for t in range(T) for h in range(n) for e in range(2 * D)}  # noqa: E731
        shared = bool(byte(k, J) & byte(o, H))
        seen[shared] += 1
        v, kc = _t(far * 2, BF16, [T, J, D]), _t(FAKE, BF16, [10, 16, J, D])
        rc = append(lib, q, k, v, o, kc, T, 8)
        assert rc == (INVALID if shared else PASSED), (T, H, J, st, sh, d, lib.pkv_last_error())
    assert min(seen.values()) > 300


# ---------------------------------------------------------------- masks
M0 = FAKE + 0x100000


@pytest.mark.parametrize("mask,pos", [(0, None), (-20, None), (None, 0), (None, 20), (None, 0x100000), (None, 0x200004), (0x100008, None),
                                      (0x200000, None), (0x300000, 0x300000 + 20)])
def test_outputs_of_a_mask(lib, mask, pos):
    """Offsets from parents (0), cu_seqlens_q (0x100000) and seq_lens (0x200000), and one output from the other."""
    a = [_t(M0, I32, [6]), _t(M0 + 0x100000, I32, [3]), _t(M0 + 0x200000, I32, [2]),
         _t(M0 + (0x400000 if mask is None else mask), I32, [6, 1]), _t(M0 + (0x500000 if pos is None else pos), I32, [6])]
    assert lib.pkv_tree_mask(*map(ptr, a), None) == INVALID
    assert b"must not overlap" in lib.pkv_last_error()
