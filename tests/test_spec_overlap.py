"""Outputs of the speculative calls that overlap what the call reads are
refused on the host (no GPU): CTAs that are still reading would see them."""
import ctypes

import pytest

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
