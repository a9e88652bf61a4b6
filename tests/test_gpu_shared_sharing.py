"""Which requests of a call read a prefix together: seen by its effect, since a
shared prefix is read through the table of the group's first request alone."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.share_ref import SharedBatch
from tests.test_gpu_shared import Dev, close

pytestmark = pytest.mark.gpu


def lose_prefixes(d, keep=()):
    """The entries of the prefix in every table but that of its group's first request, and those of `keep`, name other
    blocks: a request that reads its own table gets another result."""
    for s, (first, _, p) in enumerate(d.b.groups):
        if s != first and s not in keep:
            d.bt[s, :p // d.b.bs] = torch.arange(s, s + p // d.b.bs, dtype=torch.int32, device="cuda") % d.b.nb


def padded(d, T):
    """The batch in buffers of T rows, as a captured step has them; returns its output."""
    q = torch.full((T, *d.q.shape[1:]), float("nan"), dtype=d.q.dtype, device="cuda")
    q[:d.b.T] = d.q
    out = torch.full((T, *d.out.shape[1:]), 7.0, dtype=d.out.dtype, device="cuda")
    d.q, d.out = q, out
    return out


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bounds", [True, False])
@pytest.mark.parametrize("T", [13, 160, 2048])
def test_rows_behind_the_last_do_not_keep_requests_from_sharing(kv, bounds, T):
    b = SharedBatch([(9, 256), (4, 64)], [7 * s for s in range(13)], [1] * 13, 8, 2, 128, 16, kv, seed=61)
    d = Dev(b)
    lose_prefixes(d)
    out = padded(d, T)
    d.run(max_q=1 if bounds else 0, max_group=9 if bounds else 0)
    assert pkv.pkv_device_errors() == 0
    close(b, out[:b.T])
    assert (out[b.T:] == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bounds", [True, False])
@pytest.mark.parametrize("name,groups,new,chunks", [
    ("a chunk in a group of decodes", [(33, 128)], [1] * 16 + [300] + [1] * 16, (16,)),
    ("a chunk at the end", [(20, 128)], [1] * 19 + [257], (19,)),
    ("a chunk of another group", [(3, 64), (12, 256)], [200, 180, 190] + [1] * 12, (0, 1, 2)),
    ("a chunk alone", [(1, 0), (12, 256)], [600] + [1] * 12, (0,)),
])
def test_a_chunk_does_not_keep_decodes_from_sharing(name, groups, new, chunks, kv, bounds):
    b = SharedBatch(groups, [11 * s % 90 for s in range(len(new))], new, 8, 2, 64, 16, kv, seed=62)
    d = Dev(b)
    lose_prefixes(d, keep=chunks)  # the chunks may read theirs either way
    d.run(max_q=None if bounds else 0, max_group=None if bounds else 0)
    assert pkv.pkv_device_errors() == 0
    close(b, d.out)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bounds", [True, False])
def test_many_groups_in_buffers_with_many_more_rows(kv, bounds):
    """Runs over more requests than a warp, and than a block, looks through at a time."""
    r = np.random.default_rng(66)
    groups = [(int(g), 32 * int(p)) for g, p in zip(r.integers(1, 90, 40), r.integers(0, 6, 40))]
    B = sum(g for g, _ in groups)
    assert B > 1024
    new = [int(x) for x in r.choice([0, 1, 1, 1, 2, 5, 70], B, p=[.05, .4, .2, .2, .1, .04, .01])]
    b = SharedBatch(groups, [int(x) for x in r.integers(0, 60, B)], new, 4, 1, 64, 32, kv, seed=66)
    d = Dev(b)
    out = padded(d, 30000)
    d.run(max_q=None if bounds else 0, max_group=None if bounds else 0)
    assert pkv.pkv_device_errors() == 0
    close(b, out[:b.T])
    assert (out[b.T:] == 7.0).all()
