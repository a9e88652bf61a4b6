"""Calls with several items for each of the persistent CTAs of the tensor-core
tree kernels: the item ring, both accumulators and query buffers, references
and flags are used by one item after the other, of one, two and more tiles,
against the plain 64-bit reference."""
import numpy as np
import pytest
import torch

from tests.spec_ref import Batch
from tests.test_gpu_tree import compare, poison

pytestmark = pytest.mark.gpu


def batch(kv, q, G, D, B=96, Hkv=8, seed=70, bs=16):
    """At least 5 items a CTA of 152 (B * Hkv units): contexts of one to three tiles in random order."""
    rng = np.random.default_rng(seed)
    ctx = [int(rng.choice([5, 60, 100, 130, 200, 250, 300])) for _ in range(B)]
    return Batch(ctx, [int(rng.integers(1, q + 1)) for _ in range(B - 1)] + [q], Hkv * G, Hkv, D, bs, kv, seed=seed)


# query rows of a tile: 16, 32, 64; 128 for bf16
ROWS = [(4, 4), (8, 4), (16, 4), (20, 4)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,G", ROWS)
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_items_a_cta(kv, q, G, D):
    compare(batch(kv, q, G, D, seed=70 + q))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,G", ROWS)
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_first_key_leads(kv, q, G, D):
    """The first key of every context exceeds the others by about 12 nats (17
    powers of two): rows whose first reference does not come from it move in
    their first tile, while the output of the item before the last is read."""
    b = batch(kv, q, G, D, seed=80 + q)
    gen = torch.Generator().manual_seed(81)
    base = torch.randn((b.Hkv, D), generator=gen)
    b.q = (base.repeat_interleave(G, 0) + 0.1 * torch.randn((b.T, b.Hq, D), generator=gen)).to(b.q.dtype)
    flat = b.kc.view(-1, b.Hkv, D)
    rows = (0.05 * flat.float()).to(b.kc.dtype)
    lead = (base * (12.0 / (b.scale * (base * base).sum(1, keepdim=True))) / b.k_scale).clamp(-448, 448).to(b.kc.dtype)
    first = torch.tensor([int(b.slots(s)[0]) for s in range(b.B)])
    as_bytes = lambda t: t.view(torch.uint8)  # noqa: E731  (float8 tensors take no index)
    as_bytes(rows)[first] = as_bytes(lead)
    as_bytes(flat).copy_(as_bytes(rows))
    compare(b)


@pytest.mark.parametrize("every", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,G", ROWS)
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_values_that_are_not_finite_in_many_items(kv, q, G, D, every):
    """Drafted V rows with NaN in all items, or in every third sequence: each row that sees one shows it."""
    b = batch(kv, q, G, D, seed=90 + q)
    for s in range(0, b.B, every):
        poison(b.vc, int(b.slots(s)[b.ctx[s]]), float("nan"), 3 + s % 7)
    b.reference = lambda r=b.reference(): r  # computed once
    d = compare(b)
    want = np.isnan(b.reference()[0])
    assert want.any() and np.array_equal(torch.isnan(d.out).cpu().numpy(), want)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,q,Hq,Hkv", [(1024, 8, 32, 8), (512, 32, 32, 8), (512, 4, 64, 4)])
def test_many_sequences(B, q, Hq, Hkv, kv):
    """Large batches of small trees: up to 4,096 units."""
    rng = np.random.default_rng(B)
    b = Batch([int(c) for c in rng.integers(0, 40, B)], [q] * B, Hq, Hkv, 64, 16, kv, seed=B)
    b.reference = lambda r=b.reference(): r  # computed once
    compare(b)
    compare(b, max_q=0)
