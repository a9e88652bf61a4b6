"""Inconsistent lengths of sequences that have no row of their own are recorded
like those of the others, on every path of the tree attention."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import Batch
from tests.test_gpu_tree import Dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,q", [("f32", 5), ("bf16", 5), ("bf16", 40), ("e4m3", 5)])
def test_lengths_of_sequences_without_rows(kv, q):
    b = Batch([30, 0, 7, 0], [q, 0, 3, 0], 8, 2, 64, 16, kv, seed=5)
    want, tol = b.reference()
    d = Dev(b)
    d.run()
    assert pkv.pkv_device_errors() == 0
    d.n[1] = 16 * b.tables.shape[1] + 1  # beyond the table, no rows
    got = d.run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 4
    assert np.abs(got - want).max() <= tol
    d.n[1], d.n[3] = 0, -1  # fewer keys than rows
    got = d.run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 4
    assert np.abs(got - want).max() <= tol
    d.n[3] = 0
    d.cu[4] = d.cu[3] - 1  # rows counted backwards
    got = d.run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 4
    assert np.abs(got[:q] - want[:q]).max() <= tol


def test_many_sequences_beside_one_row():
    """f32: one CTA's threads look over all the sequences."""
    b = Batch([9] + [0] * 2999, [1] + [0] * 2999, 2, 2, 32, 16, "f32", seed=6)
    d = Dev(b)
    d.n[2999] = 10 ** 6
    got = d.run()
    assert pkv.pkv_device_errors() == 4
    want, tol = b.reference()
    assert np.abs(got.cpu().double().numpy() - want).max() <= tol
    d.n[2999] = 0
    d.run()
    assert pkv.pkv_device_errors() == 0
    assert torch.isfinite(got).all()
