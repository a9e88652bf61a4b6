"""How large a call of the speculative operators may be: what is accepted, up
to the last check before a launch (a workspace that is too short), and what
is refused.  No GPU."""
import ctypes

import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from paged_kv_cache_mapping_gb300 import build as pkv_build
from paged_kv_cache_mapping_gb300 import speculative as spec
from tests.test_abi import BF16, E4M3, F32, FAKE, I32, _t

SHORT, REFUSED, INVALID = 3, 2, 1


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return spec._lib()


def attention(lib, B, q, Hq, Hkv, max_q, D=64, dt=BF16, cdt=BF16, blocks=400, bs=16, T=None):
    """Status of a call with a workspace of no bytes: nothing is ever launched."""
    T = B * q if T is None else T
    a = [_t(FAKE, dt, [T, Hq, D]), _t(FAKE, I32, [B + 1]), _t(FAKE, I32, [B]), _t(FAKE, I32, [B, blocks]),
         _t(FAKE, cdt, [10, bs, Hkv, D]), _t(FAKE, cdt, [10, bs, Hkv, D]), _t(FAKE, I32, [T, -(-q // 32)])]
    out = _t(FAKE, F32, [T, Hq, D])
    need = ctypes.c_size_t(0)
    p = [ctypes.addressof(x) for x in a]
    assert lib.pkv_tree_attention_workspace_size(p[0], p[3], p[4], max_q, ctypes.byref(need)) == 0
    assert need.value > 0
    return lib.pkv_tree_attention(*p, 0.1, 1.0, 1.0, max_q, ctypes.addressof(out), None, 0, None)


@pytest.mark.parametrize("cdt", [BF16, E4M3])
@pytest.mark.parametrize("B,q", [(1024, 8), (512, 32), (256, 128), (512, 16), (4096, 4), (64, 2000)])
def test_ordinary_batches_are_accepted(lib, B, q, cdt):
    assert attention(lib, B, q, 32, 8, q, cdt=cdt) == SHORT, lib.pkv_last_error()
    assert attention(lib, B, q, 64, 8, q, cdt=cdt) == SHORT, lib.pkv_last_error()
    assert attention(lib, B, q, 32, 8, 0, cdt=cdt) == SHORT, lib.pkv_last_error()


def test_rows_are_numbered_in_32_bits(lib):
    # 2^30 rows in all, and one token more
    assert attention(lib, 8, 8, 32, 8, 8, T=1 << 25) == SHORT, lib.pkv_last_error()
    assert attention(lib, 8, 8, 32, 8, 8, T=(1 << 25) + 1) == REFUSED
    assert b"2^30" in lib.pkv_last_error()


@pytest.mark.parametrize("left,status", [(0, INVALID), (128, INVALID), (129, INVALID), (255, INVALID), (256, SHORT)])
def test_keys_are_numbered_in_32_bits(lib, left, status):
    """The kernels look two tiles of 128 keys past a sequence's end: that must not wrap."""
    last = (2 ** 31 - 1 - left) + 127 + 127  # the largest key number: a tile's last, of a tile that starts within 127
    assert status == INVALID or last < 2 ** 31
    assert attention(lib, 1, 8, 32, 8, 8, blocks=2 ** 31 - 1 - left, bs=1) == status, lib.pkv_last_error()


def test_a_tensor_of_too_many_dimensions_is_described_by_the_four_it_holds(lib):
    a = [_t(FAKE, I32, [6]), _t(FAKE, I32, [3]), _t(FAKE, I32, [2]), _t(FAKE, I32, [6, 1]), _t(FAKE, I32, [6])]
    for ndim in (5, 1000, 2 ** 31 - 1):
        a[0].ndim = ndim
        assert lib.pkv_tree_mask(*map(ctypes.addressof, a), None) == INVALID
        assert lib.pkv_last_error() == b"parents (i32, shape [6, 0, 0, 0, ..]): expected 1 dimensions"


def test_bounds_of_nodes_beyond_32_bits_are_refused(lib):
    i = torch.zeros(1, dtype=torch.int32)
    for n in (2 ** 31, 2 ** 32 + 8):
        with pytest.raises(pkv.PkvError, match="max_q_len beyond int32"):
            pkv.pkv_tree_attention_workspace_size(i, i, i, n)


@pytest.mark.gpu
def test_the_workspace_follows_the_bound_of_nodes():
    q = torch.zeros((64, 8, 128), dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros((4, 400), dtype=torch.int32, device="cuda")
    kc = torch.zeros((1, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    size = lambda n: pkv.pkv_tree_attention_workspace_size(q, bt, kc, n)  # noqa: E731
    assert 0 < size(1) < size(8) <= size(64) == size(0) == size(-2 ** 40) == size(2 ** 31 - 1)
