"""Trees wide enough for 128-row tiles (more than 64 query rows for each KV
head): odd sizes around the tiles, masks, scores that move a row's reference
late, pages out of range, and scales that are not positive, against the plain
64-bit reference."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import Batch, tree_attention
from tests.test_gpu_tree import Dev, compare, poison

pytestmark = pytest.mark.gpu

SHAPES = [  # ctx, q_lens, Hq, Hkv, D, bs
    ([300], [17], 8, 2, 128, 16),                          # 68 rows
    ([0, 127, 128, 129], [32, 1, 31, 20], 8, 2, 128, 16),  # 128
    ([1000, 0, 2100], [26, 5, 13], 15, 3, 64, 12),         # 130
    ([2000, 90], [33, 64], 8, 2, 128, 8),                  # 132 and 256
    ([383, 255, 700], [65, 1, 3], 8, 2, 128, 16),          # 260: a row tile of four, and short ones beside it
    ([100], [129], 3, 3, 64, 7),                           # 129
    ([640, 1], [100, 2], 8, 1, 64, 32),                    # 800
    ([5000], [40], 4, 1, 128, 1),                          # 160, one slot a page
    ([70, 3000, 12], [1, 2, 40], 20, 4, 64, 24),           # 200
    ([0], [257], 1, 1, 128, 16),                           # 257, no context
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_sizes(shape):
    compare(Batch(*SHAPES[shape], kv="bf16", seed=300 + shape))


@pytest.mark.parametrize("q", [20, 40])
def test_outputs_and_strides(q):
    b = Batch([700, 33, 2500], [q, 20, 2], 8, 2, 128, 16, "bf16", seed=31)
    f = Dev(b).run().clone()
    assert torch.equal(Dev(b, torch.bfloat16).run(), f.to(torch.bfloat16))
    for dtype in (torch.float32, torch.bfloat16):  # rows on 8 bytes only (the tensor itself on 16)
        o = torch.full((b.T, b.Hq + 2, 130 if dtype == torch.float32 else 132), 3.0, dtype=dtype, device="cuda")
        Dev(b).run(out=o[:, :8, :128])
        assert torch.equal(o[:, :8, :128], f.to(dtype))
        assert (o[:, 8:] == 3).all() and (o[:, :, 128:] == 3).all()


@pytest.mark.parametrize("q", [[30, 12, 32, 5], [40, 64, 33, 5]])
def test_general_masks(q):
    b = Batch([0, 0, 140, 300], q, 8, 2, 64, 16, "bf16", seed=32)
    rng = np.random.default_rng(2)
    b.mask = rng.integers(-2 ** 31, 2 ** 31, b.mask.shape, dtype=np.int64).astype(np.int32)  # bits past q_s too
    empty = [0, 3, q[0] + 4]
    b.mask[empty] = 0
    d = compare(b)
    assert (d.out[empty] == 0).all()  # no context, no bits


@pytest.mark.parametrize("q", [25, 50])
def test_masked_values_do_not_leak(q):
    b = Batch([150, 0, 64], [q, 9, 3], 8, 2, 128, 16, "bf16", seed=33)
    used = torch.zeros(b.nb * b.bs, dtype=torch.bool)
    for s in range(b.B):
        used[torch.from_numpy(b.slots(s))] = True
    for c in (b.kc, b.vc):
        poison(c, ~used, float("nan"))
    for s, node, v in ((0, 4, float("nan")), (1, 2, float("inf"))):
        poison(b.vc, int(b.slots(s)[b.ctx[s] + node]), v, s * 3)
    poison(b.kc, int(b.slots(0)[b.ctx[0] + 7]), float("nan"))
    for dtype in (torch.float32, torch.bfloat16):
        d = Dev(b, dtype)
        d.run()
        want, _ = b.reference()
        assert not np.isfinite(want).all() and np.isfinite(want).any()
        assert torch.equal(torch.isnan(d.out).cpu(), torch.from_numpy(np.isnan(want)))
    compare(b)


@pytest.mark.parametrize("q", [18, 40])
def test_large_and_rising_scores(q):
    b = Batch([900, 400], [q, 18], 8, 2, 128, 16, "bf16", seed=34)
    for s in range(b.B):
        rows = torch.from_numpy(b.slots(s))
        up = torch.linspace(0.05, 12.0, len(rows))[:, None, None]
        b.kc.view(-1, b.Hkv, b.D)[rows] = (b.kc.float().view(-1, b.Hkv, b.D)[rows] * up).to(b.kc.dtype)
    b.q[::3] *= 20.0
    b.q[1::5] *= 2.0 ** -20
    b.q[2::7] = 0.0
    compare(b)


@pytest.mark.parametrize("q", [4, 14, 20, 40])
def test_large_values_stay_finite(q):
    """Values near 2^100 times scores of ten powers of two: no partial sum may leave the type."""
    b = Batch([700, 40], [q, 3], 8, 2, 128, 16, "bf16", seed=39)
    b.q *= 2
    big = 2.0 ** 100
    ref, tol = b.reference()
    b.vc = (b.vc.float() * big).to(torch.bfloat16)
    got = Dev(b).run().cpu().double().numpy() / big
    assert pkv.pkv_device_errors() == 0
    assert np.abs(got - ref).max() <= tol  # a power of two scales everything exactly


@pytest.mark.parametrize("q", [20, 40])
@pytest.mark.parametrize("scale", [-0.09, 0.0])
def test_scales_that_are_not_positive(q, scale):
    b = Batch([400, 60], [q, 6], 8, 2, 128, 16, "bf16", seed=35)
    b.scale = scale
    compare(b)


@pytest.mark.parametrize("q", [20, 40])
def test_pages_out_of_range(q):
    """Nothing of a whole tile, and of the first one, is there."""
    b = Batch([500, 300], [q, 9], 8, 2, 64, 16, "bf16", seed=36)
    _, tol = b.reference()
    d = Dev(b)
    d.bt[0, :9], d.bt[0, 16:24], d.bt[1, 2] = b.nb, -1, b.nb + 5
    got = d.run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 2
    for s, lost in ((0, list(range(9)) + list(range(16, 24))), (1, [2])):
        k, v = b.rows(s)
        keep = np.ones(b.n[s], bool)
        for x in lost:
            keep[16 * x:16 * x + 16] = False
        a = b.cu[s]
        rows = slice(a, a + b.q_lens[s])
        ref, _ = tree_attention(b.q[rows].double().numpy(), k[keep], v[keep], b.mask[rows], b.scale)
        assert np.abs(got[rows] - ref).max() <= tol


def test_bad_lengths_beside_good_ones():
    b = Batch([200, 100, 300], [40, 33, 50], 8, 2, 128, 16, "bf16", seed=37)
    want, tol = b.reference()
    d = Dev(b)
    d.n[1] = 3  # fewer keys than rows
    got = d.run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 4
    assert (got[40:73] == 7.0).all()
    assert np.abs(got[:40] - want[:40]).max() <= tol and np.abs(got[73:] - want[73:]).max() <= tol


@pytest.mark.parametrize("q", [20, 64])
def test_repeats_graphs_and_streams(q):
    b = Batch([3800, 60, 700], [q, 3, 30], 8, 2, 128, 16, "bf16", seed=38)
    d = Dev(b)
    want = d.run().clone()
    ws = torch.empty(pkv.pkv_tree_attention_workspace_size(d.q, d.bt, d.kc, b.max_q), dtype=torch.uint8, device="cuda")
    for _ in range(10):
        assert torch.equal(d.run(workspace=ws), want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run(workspace=ws, out=out)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    sides = [torch.cuda.Stream() for _ in range(3)]
    res = []
    torch.cuda.synchronize()
    for _ in range(3):
        for s in sides:
            with torch.cuda.stream(s):
                res.append(d.run(out=torch.empty_like(want)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in res)
    # the other sequences change nothing
    d.n[1:] = torch.tensor([5, 321], dtype=torch.int32)
    d.q[q:] *= -3.0
    assert torch.equal(d.run()[:q], want[:q])
    assert pkv.pkv_device_errors() == 0
