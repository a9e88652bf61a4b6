"""What the speculative decoding entry points refuse on the host, before any
CUDA call, and the angles that pkv_rope_init makes (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from paged_kv_cache_mapping_gb300 import build as pkv_build
from paged_kv_cache_mapping_gb300 import speculative as spec
from tests.spec_ref import frequencies
from tests.test_abi import BF16, E4M3, F32, FAKE, I32, I64, _t

r = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return spec._lib()


def ptr(x):
    return ctypes.addressof(x) if x is not None else None


# ---------------------------------------------------------------- rope_init
@pytest.mark.parametrize("rot", [2, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor,L", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                              ("by_parts", 16.0, 4096), ("smooth", 8.0, 8192), ("linear", 0.05, 0)])
def test_rope_angles(lib, rot, scaling, factor, L):
    f, amp = frequencies(rot, 10000.0, scaling, factor, L)
    rope = pkv.pkv_rope_init(rot, 10000.0, True, scaling, factor, L)
    assert rope.rot_dim == rot and rope.interleaved == 1
    assert abs(rope.amplitude - amp) <= amp * 2.0 ** -23
    want = (f / (2 * np.pi)) % 1.0
    got = np.array([rope.turns[i] / 2.0 ** 64 for i in range(rot // 2)])
    # pow, a division or two and the blend: a few fp64 roundings of f / 2 pi
    assert (np.abs(got - want) <= 16 * 2.0 ** -53 * np.maximum(f / (2 * np.pi), 2.0 ** -11)).all()
    assert pkv.pkv_rope_init(rot, attention_factor=0.75).amplitude == 0.75


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=258), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.0), dict(scaling="ntk", factor=float("inf")),
                                dict(scaling="by_parts", factor=2.0), dict(scaling="smooth", factor=2.0),
                                dict(scaling="by_parts", factor=2.0, original_max_position=100, fast=1.0, slow=2.0),
                                dict(scaling="other"), dict(attention_factor=-1.0)])
def test_rope_init_refusals(lib, kw):
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_rope_init(**{"rot_dim": 64, **kw})
    assert e.value.status == 1


# ---------------------------------------------------------------- rope_append
def rope_args(T=4, Hq=8, Hkv=2, D=64, dt=BF16, cdt=BF16):
    return dict(q=_t(FAKE, dt, [T, Hq, D]), k=_t(FAKE, dt, [T, Hkv, D]), v=_t(FAKE, dt, [T, Hkv, D]),
                pos=_t(FAKE, I32, [T]), slots=_t(FAKE, I64, [T]), o=_t(FAKE + 0x100000, dt, [T, Hq, D]),
                kc=_t(FAKE, cdt, [10, 16, Hkv, D]), vc=_t(FAKE, cdt, [10, 16, Hkv, D]), ks=1.0, vs=1.0, rot=64)


@pytest.mark.parametrize("change,status", [
    (dict(q=_t(FAKE, BF16, [4, 8, 32])), 1), (dict(q=_t(FAKE, F32, [4, 8, 64])), 1),
    (dict(k=_t(FAKE, BF16, [4, 3, 64])), 1), (dict(v=_t(FAKE, BF16, [3, 2, 64])), 1),
    (dict(pos=_t(FAKE, F32, [4])), 1), (dict(pos=_t(FAKE, I32, [5])), 1), (dict(pos=_t(FAKE, I32, [4], [2])), 1),
    (dict(slots=_t(FAKE, I32, [3])), 1), (dict(o=_t(FAKE, BF16, [4, 8, 64], [1024, 64, 1])), 1),
    (dict(o=_t(FAKE + 2, BF16, [4, 8, 64])), 1), (dict(k=_t(FAKE, BF16, [4, 2, 64], [130, 64, 1])), 1),
    (dict(q=_t(FAKE, BF16, [4, 8, 64], [1024, 128, 2])), 1), (dict(rot=128), 1), (dict(rot=None), 1),
    (dict(kc=_t(FAKE, F32, [10, 16, 2, 64]), vc=_t(FAKE, F32, [10, 16, 2, 64])), 2),
    (dict(kc=_t(FAKE, E4M3, [10, 16, 2, 64]), vc=_t(FAKE, E4M3, [10, 16, 2, 64]), ks=0.0), 1),
    (dict(kc=_t(FAKE, E4M3, [10, 16, 2, 64]), vc=_t(FAKE, E4M3, [10, 16, 2, 64]), vs=float("inf")), 1),
])
def test_rope_append_refusals(lib, change, status):
    a = {**rope_args(), **change}
    rope = pkv.pkv_rope_init(a["rot"]) if a["rot"] else pkv.Rope()
    rc = lib.pkv_rope_append(ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["pos"]), ptr(a["slots"]), rope, ptr(a["o"]),
                             ptr(a["kc"]), ptr(a["vc"]), a["ks"], a["vs"], None)
    assert rc == status, lib.pkv_last_error()
    assert lib.pkv_last_error() != b""


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("change", [
    dict(parents=_t(FAKE, I64, [6])), dict(parents=_t(FAKE, I32, [6], [2])), dict(cu=_t(FAKE, I32, [2])),
    dict(mask=_t(FAKE, I32, [5, 1])), dict(mask=_t(FAKE, I64, [6, 1])), dict(mask=_t(FAKE, I32, [6, 0])),
    dict(mask=_t(FAKE, I32, [6, 2], [4, 2])), dict(mask=_t(FAKE, I32, [6, 2], [1, 1])), dict(pos=_t(FAKE, I32, [5])),
    dict(pos=None)])
def test_tree_mask_refusals(lib, change):
    a = {**dict(parents=_t(FAKE, I32, [6]), cu=_t(FAKE, I32, [3]), sl=_t(FAKE, I32, [2]), mask=_t(FAKE, I32, [6, 1]),
                pos=_t(FAKE, I32, [6])), **change}
    assert lib.pkv_tree_mask(ptr(a["parents"]), ptr(a["cu"]), ptr(a["sl"]), ptr(a["mask"]), ptr(a["pos"]), None) == 1


# ---------------------------------------------------------------- attention
def tree_args(T=6, Hq=8, Hkv=2, D=64, dt=BF16, cdt=BF16, W=1, max_q=3):
    return dict(q=_t(FAKE, dt, [T, Hq, D]), cu=_t(FAKE, I32, [3]), sl=_t(FAKE, I32, [2]), bt=_t(FAKE, I32, [2, 5]),
                kc=_t(FAKE, cdt, [10, 16, Hkv, D]), vc=_t(FAKE, cdt, [10, 16, Hkv, D]), mask=_t(FAKE, I32, [T, W]),
                scale=0.1, ks=1.0, vs=1.0, max_q=max_q, o=_t(FAKE, F32, [T, Hq, D]), ws=1 << 34)


@pytest.mark.parametrize("change,status", [
    (dict(q=_t(FAKE, BF16, [6, 7, 64]), o=_t(FAKE, F32, [6, 7, 64])), 1), (dict(o=_t(FAKE, F32, [6, 8, 32])), 1),
    (dict(o=_t(FAKE, I32, [6, 8, 64])), 1), (dict(mask=_t(FAKE, I32, [5, 1])), 1), (dict(mask=_t(FAKE, F32, [6, 1])), 1),
    (dict(max_q=33), 1), (dict(mask=None), 1), (dict(bt=_t(FAKE, I32, [3, 5])), 1), (dict(cu=_t(FAKE, I32, [2])), 1),
    (dict(scale=float("nan")), 1), (dict(q=_t(FAKE + 2, BF16, [6, 8, 64])), 1),
    (dict(q=_t(FAKE, F32, [6, 8, 64])), 2),
    (dict(q=_t(FAKE, BF16, [6, 8, 96]), o=_t(FAKE, F32, [6, 8, 96]), kc=_t(FAKE, BF16, [10, 16, 2, 96]),
          vc=_t(FAKE, BF16, [10, 16, 2, 96])), 2),
    (dict(kc=_t(FAKE, BF16, [1 << 26, 16, 2, 64]), vc=_t(FAKE, BF16, [1 << 26, 16, 2, 64])), 2),
    (dict(kc=_t(FAKE, E4M3, [10, 16, 2, 64]), vc=_t(FAKE, E4M3, [10, 16, 2, 64]), ks=-1.0), 1),
])
def test_tree_attention_refusals(lib, change, status):
    a = {**tree_args(), **change}
    rc = lib.pkv_tree_attention(ptr(a["q"]), ptr(a["cu"]), ptr(a["sl"]), ptr(a["bt"]), ptr(a["kc"]), ptr(a["vc"]),
                                ptr(a["mask"]), a["scale"], a["ks"], a["vs"], a["max_q"], ptr(a["o"]), FAKE, a["ws"], None)
    assert rc == status, lib.pkv_last_error()
    assert lib.pkv_last_error() != b""


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("change", [
    dict(acc=_t(FAKE, I64, [2, 4])), dict(acc=_t(FAKE, I32, [3, 4])), dict(acc=_t(FAKE, I32, [2, 4], [8, 2])),
    dict(lens=_t(FAKE, I32, [3])), dict(bt=_t(FAKE, I32, [2, 0])), dict(kc=_t(FAKE, BF16, [10, 16, 2, 60])),
    dict(new=_t(FAKE, I32, [2])), dict(new=_t(FAKE + 4, I32, [2])), dict(new=_t(FAKE + 64, I64, [2])),
    dict(kc=_t(FAKE, BF16, [10, 16, 2, 60]), vc=_t(FAKE, BF16, [10, 16, 2, 60]))])
def test_tree_commit_refusals(lib, change):
    a = {**dict(acc=_t(FAKE, I32, [2, 4]), lens=_t(FAKE, I32, [2]), cu=_t(FAKE, I32, [3]), sl=_t(FAKE, I32, [2]),
                bt=_t(FAKE, I32, [2, 5]), kc=_t(FAKE, BF16, [10, 16, 2, 64]), vc=_t(FAKE, BF16, [10, 16, 2, 64]),
                new=None), **change}
    assert lib.pkv_tree_commit(ptr(a["acc"]), ptr(a["lens"]), ptr(a["cu"]), ptr(a["sl"]), ptr(a["bt"]), ptr(a["kc"]),
                               ptr(a["vc"]), ptr(a["new"]), None) == 1


def test_binding_refuses_cpu_tensors_and_bad_types():
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: pkv.pkv_tree_mask(i, i, i, 1),
                 lambda: pkv.pkv_tree_commit(i.view(1, 2), i[:1], i, i[:1], i.view(1, 2), i, i)):
        with pytest.raises(pkv.PkvError):
            call()
    with pytest.raises(TypeError):
        pkv.pkv_tree_mask([0], i, i, 1, tree_mask=i, positions=i)
