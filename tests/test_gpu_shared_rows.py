"""Shared attention against 64 bits with a bound for each element: rows of many
keys, whose outputs are small."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.share_ref import SharedBatch
from tests.share_rows import LONG, reference
from tests.test_gpu_shared import SHAPES, Dev

pytestmark = pytest.mark.gpu


def check(b, bounds):
    want, bound = reference(b)
    for max_q, max_group in bounds:
        d = Dev(b)
        d.run(max_q=max_q, max_group=max_group)
        assert pkv.pkv_device_errors() == 0
        err = np.abs(d.out.cpu().double().numpy() - want)
        worst = float((err / np.maximum(bound, 1e-300)).max())
        assert worst <= 1.0, f"{worst:.3f} of the bound, at {np.unravel_index((err / bound).argmax(), err.shape)}"


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(LONG))
def test_long(name, kv):
    b = SharedBatch(*LONG[name], kv=kv, seed=82)
    check(b, [(b.max_q, b.max_group), (0, 0)])


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("shape", [0, 2, 3, 5, 7, 11])
def test_shapes(shape, kv):
    b = SharedBatch(*SHAPES[shape], kv=kv, seed=83)
    check(b, [(b.max_q, b.max_group), (0, 0)])


def test_a_batch_in_padded_buffers():
    b = SharedBatch([(6, 16384)], [64 * s for s in range(6)], [1] * 6, 8, 2, 64, 16, "e4m3", seed=84)
    want, bound = reference(b)
    d = Dev(b)
    q = torch.zeros((2048, 8, 64), dtype=torch.bfloat16, device="cuda")
    q[:b.T] = d.q
    out = torch.full((2048, 8, 64), 7.0, device="cuda")
    for max_q in (1, 0):
        d.run(q=q, out=out, max_q=max_q, max_group=0)
        assert (np.abs(out[:b.T].cpu().double().numpy() - want) <= bound).all()
        assert (out[b.T:] == 7.0).all()
