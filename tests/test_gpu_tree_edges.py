"""Calls that the header allows and that lie at the edges: many query heads for
one KV head, block sizes beyond a tile, scales that are not positive on every
tile width, query rows that are not finite, empty paths."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import Batch
from tests.test_gpu_tree import Dev, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,q", [(300, 1, [3, 1]), (129, 1, [1, 5]), (130, 2, [1, 1])])
def test_many_query_heads_for_a_kv_head(Hq, Hkv, q, kv):
    compare(Batch([300, 90], q, Hq, Hkv, 64, 16, kv, seed=Hq))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("bs", [256, 1000, 129, 4100])
def test_blocks_longer_than_a_tile(bs, kv):
    compare(Batch([1500, 0, 260], [5, 2, 20], 8, 2, 64, bs, kv, seed=bs, slack=1))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("q", [4, 8, 16, 20])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30])
def test_scales(scale, q, kv):
    b = Batch([400, 60], [q, 3], 8, 2, 128, 16, kv, seed=41)
    b.scale = scale
    compare(b)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("q", [4, 20, 40])
def test_query_rows_that_are_not_finite(q, kv):
    """NaN in a head of a node reaches that head's row alone."""
    b = Batch([400, 60], [q, 3], 8, 2, 128, 16, kv, seed=42)
    want, tol = b.reference()
    b.q[1, 3, 7] = float("nan")
    b.q[q, 0] = float("nan")
    got = Dev(b).run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 0
    hit = np.zeros(got.shape[:2], bool)
    hit[1, 3] = hit[q, 0] = True
    assert np.isnan(got[hit]).all()
    assert np.abs(got[~hit] - want[~hit]).max() <= tol


@pytest.mark.parametrize("A", [0, 3])
def test_empty_paths(A):
    b = Batch([20, 0, 5], [4, 2, 0], 2, 2, 64, 16, "bf16", seed=43)
    d = Dev(b)
    kc = d.kc.clone()
    new = pkv.pkv_tree_commit(torch.zeros((3, A), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                              d.cu, d.n, d.bt, d.kc, d.vc)
    assert pkv.pkv_device_errors() == 0
    assert new.tolist() == b.ctx
    assert torch.equal(d.kc, kc)
