"""What the entry points for requests that share prompts refuse on the host,
before any CUDA call, and the plain references against hand-worked steps (no GPU)."""
import ctypes

import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from paged_kv_cache_mapping_gb300 import build as pkv_build
from paged_kv_cache_mapping_gb300 import speculative as spec
from tests import share_ref
from tests.test_abi import BF16, E4M3, F32, FAKE, I32, I64, _t

PASSED = 4  # no GPU here: the first CUDA call after the checks fails


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return spec._lib()


def ptr(x):
    return ctypes.addressof(x) if x is not None else None


def at(k, dtype, shape, stride=None):
    return _t(FAKE + 0x100000 * k, dtype, shape, stride)


def table_args(B=3, T=7, W=5, F=20):
    return dict(old=at(1, I32, [B]), new=at(2, I32, [B]), shared=at(3, I32, [B]), bs=16, bt=at(4, I32, [B, W]), free=at(5, I32, [F]),
                count=at(6, I32, [1]), left=at(7, I32, [1]), cu=at(8, I32, [B + 1]), slots=at(9, I32, [T]), pos=at(10, I32, [T]))


def step_tables(lib, a):
    return lib.pkv_step_tables(ptr(a["old"]), ptr(a["new"]), ptr(a["shared"]), a["bs"], ptr(a["bt"]), ptr(a["free"]), ptr(a["count"]),
                               ptr(a["left"]), ptr(a["cu"]), ptr(a["slots"]), ptr(a["pos"]), None)


@pytest.mark.parametrize("change,status", [
    (dict(old=None), 1), (dict(old=at(1, I64, [3])), 1), (dict(new=at(2, I32, [2])), 1), (dict(new=at(2, I32, [3], [2])), 1),
    (dict(shared=at(3, I32, [4])), 1), (dict(shared=at(3, BF16, [3])), 1), (dict(bs=0), 1), (dict(bs=-4), 1),
    (dict(bt=at(4, I32, [2, 5])), 1), (dict(bt=at(4, I32, [3, 0])), 1), (dict(bt=at(4, I32, [3, 5], [10, 2])), 1),
    (dict(bt=at(4, I32, [3, 5], [4, 1])), 1), (dict(bt=at(4, I64, [3, 5])), 1), (dict(bs=1 << 30), 1),
    (dict(free=at(5, I64, [20])), 1), (dict(free=None), 1), (dict(free=at(5, I32, [20], [2])), 1), (dict(count=at(6, I32, [2])), 1),
    (dict(count=at(6, I64, [1])), 1), (dict(left=None), 1), (dict(left=at(7, I32, [0])), 1), (dict(cu=at(8, I32, [3])), 1),
    (dict(slots=at(9, BF16, [7])), 1), (dict(slots=at(9, I64, [8])), 1), (dict(slots=None), 1), (dict(pos=at(10, I32, [6])), 1),
    (dict(pos=at(10, I64, [7])), 1),
    # outputs over inputs and over each other
    (dict(left=at(1, I32, [1])), 1), (dict(cu=at(2, I32, [4])), 1), (dict(slots=at(4, I64, [7])), 1), (dict(pos=at(9, I32, [7])), 1),
    (dict(free=at(4, I32, [20])), 1), (dict(slots=at(3, I32, [7])), 1), (dict(cu=at(6, I32, [4])), 1), (dict(left=at(5, I32, [1])), 1),
    (dict(bt=at(1, I32, [3, 5])), 1), (dict(free=at(6, I32, [20])), 1),
    # more requests than a call takes
    (table_args(B=8193), 2),
    # what passes: no shared blocks, no positions, the count in place, nothing to do
    ({}, PASSED), (dict(shared=None), PASSED), (dict(pos=None), PASSED), (dict(left=at(6, I32, [1])), PASSED), (table_args(B=8192), PASSED),
    (table_args(B=0, T=0), PASSED), (dict(slots=at(9, I64, [7])), PASSED), (dict(free=at(5, I32, [0])), PASSED),
])
def test_step_tables_refusals(lib, change, status):
    if status == PASSED and torch.cuda.is_available():
        pytest.skip("what passes the checks would be launched")
    assert step_tables(lib, {**table_args(), **change}) == status, lib.pkv_last_error()
    assert lib.pkv_last_error() != b""


@pytest.mark.parametrize("change,status", [
    (dict(cu=at(1, I32, [3])), 1), (dict(n=at(2, I64, [3])), 1), (dict(n=None), 1), (dict(bt=at(3, I32, [4, 5])), 1), (dict(bs=0), 1),
    (dict(least=0), 1), (dict(least=-7), 1), (dict(g=at(4, I32, [3, 2])), 1), (dict(g=at(4, I32, [4, 3])), 1), (dict(g=at(4, I64, [3, 3])), 1),
    (dict(g=at(4, I32, [3, 3], [4, 1])), 1), (dict(g=None), 1), (dict(g=at(2, I32, [3, 3])), 1), (dict(g=at(3, I32, [3, 3])), 1),
    (dict(g=at(1, I32, [3, 3])), 1), (dict(bs=1 << 30), 1),
    (dict(cu=at(1, I32, [8194]), n=at(2, I32, [8193]), bt=at(3, I32, [8193, 5]), g=at(4, I32, [8193, 3])), 2), ({}, PASSED),
])
def test_shared_prefixes_refusals(lib, change, status):
    if status == PASSED and torch.cuda.is_available():
        pytest.skip("what passes the checks would be launched")
    a = {**dict(cu=at(1, I32, [4]), n=at(2, I32, [3]), bt=at(3, I32, [3, 5]), bs=16, least=16, g=at(4, I32, [3, 3])), **change}
    rc = lib.pkv_shared_prefixes(ptr(a["cu"]), ptr(a["n"]), ptr(a["bt"]), a["bs"], a["least"], ptr(a["g"]), None)
    assert rc == status, lib.pkv_last_error()


def test_binding_refuses_cpu_tensors_and_bad_numbers():
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: pkv.pkv_step_tables(i, i, i.view(1, 2), 16, i, i[:1], i, i), lambda: pkv.pkv_shared_prefixes(i, i, i.view(1, 2), 16)):
        with pytest.raises(pkv.PkvError):
            call()
    with pytest.raises(TypeError):
        pkv.pkv_step_tables([0], i, i.view(1, 2), 16, i, i[:1], i, i)


# ---------------------------------------------------------------- the references
def test_reference_of_a_step_by_hand():
    # blocks of 4: request 0 decodes into a new block, 1 is done, 2 loses two drafted tokens, 3 is admitted behind a shared block
    tables = [[7, -1, -1], [1, 2, -1], [3, 4, 5], [9, -1, -1]]
    out = share_ref.step_tables([4, 6, 10, 4], [5, 0, 8, 9], [0, 0, 0, 1], 4, tables, [20, 21, 22, 0, 0, 0], 3, 7)
    # the stack is 20 21 22 | 1 2 | 5: taken are 5 (request 0), then 2 and 1 (request 3)
    assert out[0] == [[7, 5, -1], [1, 2, -1], [3, 4, 5], [9, 2, 1]]
    assert out[1] == [20, 21, 22, 0, 0, 0] and out[2] == 3
    assert out[3] == [0, 1, 1, 1, 6]
    assert out[4] == [20, 8, 9, 10, 11, 4, -1] and out[5] == [4, 4, 5, 6, 7, 8, 0] and out[6] == 0


def test_reference_of_refused_steps():
    tables = [[7, -1]]
    assert share_ref.step_tables([4], [9], [0], 4, tables, [5], 1, 5)[6] == 4  # beyond the table: takes no part
    out = share_ref.step_tables([4], [8], [0], 4, tables, [5], 0, 4)
    assert out[6] == 32 and out[0] == tables and out[3] == [0, 0] and out[4] == [-1] * 4
    assert share_ref.step_tables([4], [8], [0], 4, tables, [5], 1, 3)[6] == 4  # more rows than slots
    assert share_ref.step_tables([4], [0], [0], 4, tables, [5], 1, 0)[6] == 4  # the list cannot hold it


def test_reference_of_groups_by_hand():
    tables = [[1, 2, 3, 4, 0], [1, 2, 3, 5, 0], [1, 2, 3, 6, 0], [1, 9, 9, 9, 0], [8, 9, 9, 9, 0], [-1] * 5, [-1] * 5]
    n = [17, 16, 17, 13, 16, 16, 16]
    cu = [0, 1, 2, 3, 4, 5, 6, 7]
    # full blocks of four tokens: 4, 3, 4, 3, 3, 3, 3; common: 3, 3, 1, 0, 0, 0
    out, flags = share_ref.shared_prefixes(cu, n, tables, 4, 4)
    assert flags == 0
    assert out == [[0, 3, 12]] * 3 + [[3, 4, 0], [4, 5, 0], [5, 6, 0], [6, 7, 0]]
    assert share_ref.shared_prefixes(cu, n, tables, 4, 13)[0] == [[s, s + 1, 0] for s in range(7)]
    assert share_ref.shared_prefixes([0, 20], [5], [[1, 2]], 4, 1) == ([[0, 1, 0]], 4)


# ---------------------------------------------------------------- attention
SHORT = 3


def attention_args(T=6, Hq=8, Hkv=2, D=64, dt=BF16, cdt=BF16, B=2):
    return dict(q=at(1, dt, [T, Hq, D]), cu=at(2, I32, [B + 1]), sl=at(3, I32, [B]), bt=at(4, I32, [B, 5]), g=at(5, I32, [B, 3]),
                kc=at(6, cdt, [10, 16, Hkv, D]), vc=at(7, cdt, [10, 16, Hkv, D]), scale=0.1, ks=1.0, vs=1.0, max_q=3, max_g=6,
                o=at(8, F32, [T, Hq, D]), ws=FAKE, bytes=1 << 34)


def attention(lib, a):
    return lib.pkv_shared_attention(ptr(a["q"]), ptr(a["cu"]), ptr(a["sl"]), ptr(a["bt"]), ptr(a["g"]), ptr(a["kc"]), ptr(a["vc"]), a["scale"],
                                    a["ks"], a["vs"], a["max_q"], a["max_g"], ptr(a["o"]), a["ws"], a["bytes"], None)


@pytest.mark.parametrize("change,status", [
    (dict(q=at(1, BF16, [6, 7, 64]), o=at(8, F32, [6, 7, 64])), 1), (dict(o=at(8, F32, [6, 8, 32])), 1), (dict(o=at(8, I32, [6, 8, 64])), 1),
    (dict(g=at(5, I32, [3, 3])), 1), (dict(g=at(5, I32, [2, 2])), 1), (dict(g=at(5, I64, [2, 3])), 1), (dict(g=at(5, I32, [2, 3], [4, 1])), 1),
    (dict(g=at(5, I32, [6])), 1), (dict(g=None), 1), (dict(bt=at(4, I32, [3, 5])), 1), (dict(cu=at(2, I32, [2])), 1), (dict(sl=None), 1),
    (dict(scale=float("nan")), 1), (dict(q=at(1, BF16, [6, 8, 64], [1024, 64, 1]), o=at(8, F32, [6, 8, 64], [513, 64, 1])), 1),
    (dict(q=_t(FAKE + 2, BF16, [6, 8, 64])), 1), (dict(q=at(1, BF16, [6, 8, 64], [514, 64, 1])), 1), (dict(q=at(1, F32, [6, 8, 64])), 2),
    (dict(q=at(1, BF16, [6, 8, 96]), o=at(8, F32, [6, 8, 96]), kc=at(6, BF16, [10, 16, 2, 96]), vc=at(7, BF16, [10, 16, 2, 96])), 2),
    (dict(kc=at(6, BF16, [1 << 26, 16, 2, 64]), vc=at(7, BF16, [1 << 26, 16, 2, 64])), 2), (dict(kc=at(6, BF16, [0, 16, 2, 64]), vc=at(7, BF16, [0, 16, 2, 64])), 1),
    (dict(kc=at(6, E4M3, [10, 16, 2, 64]), vc=at(7, E4M3, [10, 16, 2, 64]), ks=-1.0), 1), (dict(vc=at(7, BF16, [10, 16, 2, 128])), 1),
    (dict(bt=at(4, I32, [2, 2 ** 27])), 1), (dict(bytes=0), SHORT), (dict(bytes=255), SHORT), (dict(ws=FAKE + 16), 1), (dict(ws=None), 1),
    ({}, PASSED), (dict(max_q=0, max_g=0), PASSED), (dict(max_q=-5, max_g=1 << 30), PASSED),
])
def test_shared_attention_refusals(lib, change, status):
    if status == PASSED and torch.cuda.is_available():
        pytest.skip("what passes the checks would be launched")
    assert attention(lib, {**attention_args(), **change}) == status, lib.pkv_last_error()
    assert lib.pkv_last_error() != b""


def workspace(lib, a):
    n = ctypes.c_size_t(0)
    assert lib.pkv_shared_attention_workspace_size(ptr(a["q"]), ptr(a["bt"]), ptr(a["kc"]), a["max_q"], a["max_g"], ctypes.byref(n)) == 0
    return n.value


def test_workspace_sizes(lib):
    """A row for each token and chunk of a prefix, one more for each, and the chunks of a request's own keys."""
    a = attention_args(T=64, Hq=32, Hkv=8, D=128, B=64)
    row = 4 * 32 * 129
    for blocks in (1, 8, 100, 100000):
        for q, g in ((1, 1), (1, 64), (0, 0)):
            n = workspace(lib, {**a, "bt": at(4, I32, [64, blocks]), "max_q": q, "max_g": g})
            assert 64 * row <= n <= (64 * 65 + 64 * 1024) * row + 256
    assert workspace(lib, {**a, "kc": at(6, F32, [10, 16, 8, 128])}) == 0  # f32 needs none
    assert workspace(lib, {**attention_args(T=0), "q": at(1, BF16, [0, 8, 64])}) == 0
    huge = {**attention_args(T=1 << 25, Hq=32, Hkv=8, D=64), "max_q": 0, "max_g": 0}
    assert workspace(lib, huge) > 0
    assert attention(lib, {**huge, "o": at(8, F32, [1 << 25, 32, 64]), "kc": at(6, BF16, [10, 16, 8, 64]), "vc": at(7, BF16, [10, 16, 8, 64]),
                           "bytes": 0}) == SHORT
    for name in ("max_q_len", "max_group_len"):
        with pytest.raises(pkv.PkvError, match=f"{name} beyond int32"):
            i = torch.zeros(1, dtype=torch.int32)
            pkv.pkv_shared_attention_workspace_size(i, i, i, **{name: 2 ** 31})
