"""Where a request stands in its group: its rows take other places of the prefix's
tiles, and get the same bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.share_ref import SharedBatch
from tests.test_gpu_shared import Dev, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq", [8, 16, 40])
def test_the_order_of_a_group_changes_no_bit(kv, Hq):
    new = [1, 3, 2, 1, 5, 1, 2, 1]
    b = SharedBatch([(8, 640)], [40 * s for s in range(8)], new, Hq, 2, 128, 16, kv, seed=64)
    d = Dev(b)
    want = d.run().clone()
    close(b, want)
    for order in ([7, 6, 5, 4, 3, 2, 1, 0], [1, 0, 2, 3, 4, 5, 6, 7], [4, 0, 5, 1, 6, 2, 7, 3]):
        e = Dev(b)
        rows = torch.cat([torch.arange(int(b.cu[s]), int(b.cu[s + 1])) for s in order]).cuda()
        e.q, e.n, e.bt = d.q[rows], d.n[order], d.bt[order]
        e.cu = torch.from_numpy(np.concatenate([[0], np.cumsum([new[s] for s in order])]).astype(np.int32)).cuda()
        assert torch.equal(e.run(), want[rows]), order
    assert pkv.pkv_device_errors() == 0
