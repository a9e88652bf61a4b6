"""Groups that the caller made: each request follows the numbers that it names
itself, whatever its neighbours name."""
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.share_ref import SharedBatch
from tests.test_gpu_shared import Dev, close
from tests.test_gpu_shared_sharing import padded

pytestmark = pytest.mark.gpu

# eight requests that all share a prefix of 128 tokens: what each of them names
GROUPS = {
    "one begins inside another": [(0, 4, 128)] * 2 + [(2, 6, 128)] * 4 + [(6, 8, 128)] * 2,
    "one lies inside another": [(0, 8, 128)] * 2 + [(2, 5, 64)] * 3 + [(0, 8, 128)] * 3,
    "each names all behind it": [(s, 8, 128) for s in range(8)],
    "prefixes by turns": [(0, 8, 128), (1, 8, 64)] * 4,
    "some alone between": [(0, 8, 128), (3, 4, 0), (0, 8, 128), (0, 8, 128), (-7, 99, 0), (0, 8, 128), (0, 8, 128), (0, 0, 0)],
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("new", [[1] * 8, [1, 3, 2, 1, 40, 1, 2, 1]])
@pytest.mark.parametrize("name", list(GROUPS))
def test_groups_that_overlap(name, new, kv):
    b = SharedBatch([(8, 128)], [20 * s for s in range(8)], new, 8, 2, 64, 16, kv, seed=71)
    for bounds in ((b.max_q, b.T), (0, 0)):
        d = Dev(b)
        d.groups.copy_(torch.tensor(GROUPS[name], dtype=torch.int32))
        d.run(*bounds)
        assert pkv.pkv_device_errors() == 0
        close(b, d.out)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1] * 8, [1, 3, 2, 1, 300, 1, 2, 1]])
@pytest.mark.parametrize("name", list(GROUPS))
def test_groups_that_overlap_in_buffers_with_many_more_rows(name, new, kv):
    b = SharedBatch([(8, 128)], [20 * s for s in range(8)], new, 8, 2, 64, 16, kv, seed=73)
    d = Dev(b)
    d.groups.copy_(torch.tensor(GROUPS[name], dtype=torch.int32))
    out = padded(d, 3000)
    d.run(0, 0)
    assert pkv.pkv_device_errors() == 0
    close(b, out[:b.T])
    assert (out[b.T:] == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [31, 33, 64, 65, 129, 300])
def test_runs_over_many_requests(kv, B):
    """Runs that end, and groups that are broken, at every place of a warp's 32 requests."""
    b = SharedBatch([(B, 64)], [s % 50 for s in range(B)], [1 + s % 2 for s in range(B)], 4, 2, 64, 16, kv, seed=72)
    d = Dev(b)
    d.run()
    want = d.out.clone()
    close(b, want)
    for at in {0, 1, 30, 31, 32, 33, 63, 64, 127, 128, 159, 160, 161, B - 1} & set(range(B)):
        e = Dev(b)
        e.groups[at] = torch.tensor([0, 0, 0], dtype=torch.int32) if at else torch.tensor([0, 1, 64], dtype=torch.int32)
        e.run()
        # request 0 names another group: the others' first request does not name theirs
        assert pkv.pkv_device_errors() == (4 if at == 0 and B > 1 else 0)
        rows = slice(int(b.cu[at]), int(b.cu[at + 1]))
        close(b, e.out, rows)
        if at:
            close(b, e.out)
        else:
            assert (e.out[int(b.cu[1]):] == 7.0).all()
