"""The speculative calls far into a large cache (element offsets beyond 32
bits) and over a very long context."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import Batch
from tests.test_gpu_tree import Dev, compare

pytestmark = pytest.mark.gpu

BLOCKS = 280000  # times 16 slots, 8 heads, 128 elements: 4.6e9 elements


@pytest.mark.parametrize("q", [8, 40])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_at_the_end_of_a_large_cache(kv, q):
    """The same rows in the last blocks of a large cache and in a small one: same bits."""
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    b = Batch([700, 20], [q, 5], 16, 8, 128, 16, kv, seed=61)
    d = Dev(b)
    first = BLOCKS - b.nb
    big = []
    for small in (d.kc, d.vc):
        c = torch.empty((BLOCKS,) + tuple(small.shape[1:]), dtype=small.dtype, device="cuda")
        c[first:].view(torch.uint8).copy_(small.view(torch.uint8))
        big.append(c)
    rope = pkv.pkv_rope_init(128)
    gen = torch.Generator().manual_seed(3)
    k = torch.randn((b.T, 8, 128), generator=gen).bfloat16().cuda()
    positions = torch.from_numpy(b.pos.astype(np.int32)).cuda()
    accepted = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    accepted[0] = torch.tensor([0, 3, 6])
    accepted[1] = torch.tensor([1, 4, 0])
    lens = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    res = []
    for kc, vc, shift in ((d.kc, d.vc, 0), (big[0], big[1], first)):
        bt = torch.where(d.bt >= 0, d.bt + shift, d.bt)
        slots = pkv.pkv_slot_mapping(d.cu, d.n, bt, 16, T=b.T)
        q2 = pkv.pkv_rope_append(d.q, k, k, positions, slots, rope, kc, vc, k_scale=b.k_scale, v_scale=b.v_scale)
        out = pkv.pkv_tree_attention(q2, d.cu, d.n, bt, kc, vc, d.mask, b.scale, torch.empty_like(d.out), k_scale=b.k_scale,
                                     v_scale=b.v_scale, max_q_len=b.max_q)
        n2 = pkv.pkv_tree_commit(accepted, lens, d.cu, d.n, bt, kc, vc)
        res.append((q2, out, n2))
    assert pkv.pkv_device_errors() == 0
    for small, far in zip(*res):
        assert torch.equal(small, far)
    for small, far in zip((d.kc, d.vc), big):
        assert torch.equal(small.view(torch.uint8), far[first:].view(torch.uint8))
    assert torch.isfinite(res[0][1]).all()


@pytest.mark.parametrize("G", [2, 40])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_context_of_600000_keys(kv, G):
    compare(Batch([600000], [2], G, 1, 64, 64, kv, seed=62))
