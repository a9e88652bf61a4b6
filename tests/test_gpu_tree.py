"""Drafted trees: masks, attention over the paged cache and the path commit
against plain 64-bit references, where they can go wrong: single tokens, long
contexts, pages that end inside a tile, rows without a visible key, values
that must not leak, bad lengths and pages, strides, streams and graphs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import Batch, tree_attention, tree_mask

pytestmark = pytest.mark.gpu


class Dev:
    """A batch on the GPU."""

    def __init__(self, b, out_dtype=torch.float32):
        c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.b = b
        self.q, self.kc, self.vc = b.q.cuda(), b.kc.cuda(), b.vc.cuda()
        self.cu, self.n, self.bt, self.mask = c(b.cu), c(np.array(b.n, np.int32)), c(b.tables), c(b.mask)
        self.parents = c(b.parents)
        self.out = torch.full((b.T, b.Hq, b.D), 7.0, dtype=out_dtype, device="cuda")

    def run(self, max_q=None, **kw):
        b = self.b
        return pkv.pkv_tree_attention(kw.pop("q", self.q), self.cu, self.n, self.bt, self.kc, self.vc, self.mask, b.scale,
                                      kw.pop("out", self.out), k_scale=b.k_scale, v_scale=b.v_scale,
                                      max_q_len=b.max_q if max_q is None else max_q, **kw)


def poison(cache, where, value, cols=slice(None)):
    """Sets rows (all heads) of a flat cache to a value, as its stored bits."""
    bits = {4: torch.int32, 2: torch.int16, 1: torch.uint8}[cache.element_size()]
    v = torch.tensor([value]).to(cache.dtype).view(bits)[0]
    cache.view(bits).view(-1, *cache.shape[2:])[where, :, cols] = v


def compare(b, flags=0, out=None, max_q=None):
    d = Dev(b)
    got = d.run(max_q=max_q) if out is None else out
    torch.cuda.synchronize()
    assert pkv.pkv_device_errors() == flags
    want, tol = b.reference()
    got = got.cpu().double().numpy()
    both = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), both)
    err = np.abs(got[both] - want[both])
    assert err.size == 0 or err.max() <= tol, f"max err {err.max():.3e}, tolerance {tol:.3e}"
    return d


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("q_lens", [[1], [16, 16], [3, 0, 40, 1, 64], [33], [130, 257], [2100]])
def test_tree_mask(q_lens):
    rng = np.random.default_rng(len(q_lens))
    n = [q + int(rng.integers(0, 50)) for q in q_lens]
    for chain in (False, True):
        parents = np.array([i - 1 if chain else int(rng.integers(-1, i)) if i else -1 for q in q_lens for i in range(q)],
                           np.int32)
        words = -(-max(q_lens) // 32) + 1
        want, pos = tree_mask(parents, q_lens, n, words)
        cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        buf = torch.full((len(parents), words + 3), -9, dtype=torch.int32, device="cuda")
        got, gp = pkv.pkv_tree_mask(torch.from_numpy(parents).cuda(), torch.from_numpy(cu).cuda(),
                                    torch.tensor(n, dtype=torch.int32).cuda(), max(q_lens), tree_mask=buf[:, :words])
        assert pkv.pkv_device_errors() == 0
        assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(gp.cpu().numpy(), pos)
        assert (buf[:, words:] == -9).all()


def test_tree_mask_bad_links_and_lengths():
    #        0: ok        1: bad links          2: q > N  3: more nodes than bits
    q_lens, n = [4, 4, 3, 40], [9, 4, 2, 50]
    parents = [-1, 0, 0, 2, -1, 1, -2, 7, -1, 0, 1] + [i - 1 for i in range(40)]
    fixed = [-1, 0, 0, 2, -1, -1, -1, -1]
    cu = torch.tensor([0, 4, 8, 11, 51], dtype=torch.int32).cuda()
    mask = torch.full((53, 1), 5, dtype=torch.int32, device="cuda")
    pos = torch.full((53,), 5, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_mask(torch.tensor(parents + [0, 0], dtype=torch.int32).cuda(), cu, torch.tensor(n, dtype=torch.int32).cuda(),
                      32, tree_mask=mask, positions=pos)
    assert pkv.pkv_device_errors() == 4
    want, wpos = tree_mask(np.array(fixed), q_lens[:2], n[:2], 1)
    assert np.array_equal(mask[:8].cpu().numpy(), want) and np.array_equal(pos[:8].cpu().numpy(), wpos)
    assert (mask[8:51] == 0).all() and (pos[8:51] == 0).all()
    assert (mask[51:] == 5).all() and (pos[51:] == 5).all()  # rows behind the last sequence


# ---------------------------------------------------------------- attention
SHAPES = [  # ctx, q_lens, Hq, Hkv, D, bs
    ([2000], [8], 32, 8, 128, 16),
    ([700, 0, 5, 1300], [8, 8, 3, 1], 8, 2, 128, 16),
    ([0, 0, 0], [1, 2, 5], 4, 4, 64, 8),
    ([127, 128, 129, 255, 256, 257], [1, 1, 1, 1, 1, 1], 4, 1, 128, 16),
    ([120, 121, 122, 250, 254], [8, 7, 6, 7, 2], 8, 4, 64, 16),
    ([300, 511, 40], [17, 64, 33], 4, 1, 128, 32),
    ([300, 77], [16, 5], 15, 3, 64, 12),
    ([513, 90], [9, 30], 7, 1, 128, 1),
    ([1030, 64], [4, 20], 6, 6, 128, 7),
    ([200, 333], [100, 47], 8, 1, 64, 64),
    ([90], [130], 2, 2, 128, 4),
    ([5000, 100], [3, 6], 4, 2, 128, 16),
    ([3000], [70], 20, 4, 64, 24),
    ([60, 250], [2, 3], 160, 2, 64, 16),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tree_attention(shape, kv):
    compare(Batch(*SHAPES[shape], kv=kv, seed=100 + shape))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_tree_attention_f32(D):
    compare(Batch([70, 0, 300], [5, 1, 33], 6, 2, D, 16, "f32", seed=D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bf16_output_is_the_rounded_f32_output(kv):
    b = Batch([700, 33, 0], [8, 20, 2], 8, 2, 128, 16, kv, seed=5)
    f = Dev(b).run().clone()
    h = Dev(b, torch.bfloat16).run()
    assert torch.equal(h, f.to(torch.bfloat16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_rows_that_see_nothing_and_general_masks(kv):
    b = Batch([0, 0, 140, 300], [6, 40, 40, 9], 8, 2, 64, 16, kv, seed=9)
    rng = np.random.default_rng(1)
    b.mask = rng.integers(-2 ** 31, 2 ** 31, b.mask.shape, dtype=np.int64).astype(np.int32)  # bits past q_s too
    b.mask[[0, 3, 10, 50]] = 0
    d = compare(b)
    assert (d.out[[0, 3, 10]] == 0).all()  # no context, no bits


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_masked_values_do_not_leak(kv):
    b = Batch([150, 0, 64], [12, 9, 3], 8, 2, 64, 16, kv, seed=13)
    bad = [float("nan")] + ([] if kv == "e4m3" else [float("inf"), -float("inf")])
    # everything outside the sequences is poison, in K and V
    used = torch.zeros(b.nb * b.bs, dtype=torch.bool)
    for s in range(b.B):
        used[torch.from_numpy(b.slots(s))] = True
    for c in (b.kc, b.vc):
        poison(c, ~used, bad[0])
    # one drafted node of each tree holds poison; only rows that see it may show it
    for s, node in ((0, 4), (1, 2)):
        slot = int(b.slots(s)[b.ctx[s] + node])
        poison(b.vc, slot, bad[s % len(bad)], s * 3)
    slot = int(b.slots(0)[b.ctx[0] + 7])
    poison(b.kc, slot, bad[0])
    d = compare(b)
    want, _ = b.reference()
    assert not np.isfinite(want).all() and np.isfinite(want).any()
    assert torch.equal(torch.isnan(d.out).cpu(), torch.from_numpy(np.isnan(want)))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_context_values_pass_through(kv):
    """A context key is seen by every row: its NaN reaches all of them."""
    b = Batch([300], [5], 4, 1, 128, 16, kv, seed=14)
    poison(b.vc, int(b.slots(0)[17]), float("nan"), 5)
    out = Dev(b).run()
    assert torch.isnan(out[:, :, 5]).all() and not torch.isnan(out[:, :, 6:]).any()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_and_rising_scores(kv):
    """Scores that climb by far more than the type's exponent along the keys,
    and rows of very different size."""
    b = Batch([900, 400], [6, 18], 8, 2, 128, 16, kv, seed=15)
    for s in range(b.B):
        rows = torch.from_numpy(b.slots(s))
        up = torch.linspace(0.05, 12.0 if kv == "bf16" else 1.0, len(rows))[:, None, None]
        b.kc.view(-1, b.Hkv, b.D)[rows] = (b.kc.float().view(-1, b.Hkv, b.D)[rows] * up).to(b.kc.dtype)
    b.q[::3] *= 20.0
    b.q[1::5] *= 2.0 ** -20
    b.q[2::7] = 0.0
    compare(b)


def test_one_dominant_key_and_many_small_ones():
    b = Batch([4000], [4], 8, 2, 128, 16, "e4m3", seed=16)
    rows = torch.from_numpy(b.slots(0))
    b.kc.view(-1, 2, 128)[rows] = (b.kc.float().view(-1, 2, 128)[rows] * 0.02).to(b.kc.dtype)
    b.kc.view(-1, 2, 128)[int(rows[2000])] = (b.q[0, 0].float().sign() * 300).to(b.kc.dtype)
    compare(b)


def test_wide_masks_and_the_other_sequences_change_nothing():
    b = Batch([3000, 20, 500], [8, 1, 40], 8, 2, 128, 16, "bf16", seed=17, mask_words=5)
    a = Dev(b).run().clone()
    assert torch.equal(a, Dev(b).run(max_q=40))
    compare(b, out=Dev(b).run(max_q=0))  # unknown: every row could be one tree's
    compare(b, out=Dev(b).run(max_q=160))
    # the other sequences get other lengths, queries and values
    d = Dev(b)
    d.n[1:] = torch.tensor([1, 321], dtype=torch.int32)
    d.q[8:] *= -3.0
    d.mask[8:] = -1
    d.vc.view(-1, 2, 128)[torch.from_numpy(b.slots(2)).cuda()] = 9.0
    assert torch.equal(a[:8], d.run()[:8])
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_layout_changes_nothing(kv):
    """The same logical rows on pages of other sizes and places: same bits."""
    first = None
    for bs in (16, 1, 4, 8, 12, 64):
        b = Batch([610, 33], [9, 17], 8, 2, 128, bs, kv, seed=18)
        if first is None:
            first, q, mask = b, b.q, b.mask
        for s in range(2):
            sl = torch.from_numpy(b.slots(s))
            fl = torch.from_numpy(first.slots(s))
            for mine, theirs in ((b.kc, first.kc), (b.vc, first.vc)):  # as bytes: float8 tensors take no index
                rows = lambda c: c.view(torch.uint8).view(-1, 2 * 128 * c.element_size())  # noqa: E731
                rows(mine)[sl] = rows(theirs)[fl]
        b.q, b.mask = q, mask
        got = Dev(b).run().clone()
        if bs == 16:
            want = got
        assert torch.equal(got, want), bs


def test_strided_queries_and_outputs():
    b = Batch([300, 20], [8, 5], 8, 2, 128, 16, "bf16", seed=19)
    d = Dev(b)
    want = d.run().clone()
    wide_q = torch.zeros((b.T, b.Hq + 3, 136), dtype=torch.bfloat16, device="cuda")
    wide_q[:, 2:10, :128] = d.q
    wide_o = torch.full((b.T, b.Hq + 2, 132), 3.0, device="cuda")
    d.run(q=wide_q[:, 2:10, :128], out=wide_o[:, 1:9, :128])
    assert torch.equal(wide_o[:, 1:9, :128], want)
    assert (wide_o[:, 0] == 3).all() and (wide_o[:, 9:] == 3).all() and (wide_o[:, :, 128:] == 3).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_bad_pages_and_lengths(kv):
    b = Batch([200, 100, 100, 100, 60], [5, 4, 3, 40, 2], 8, 2, 64, 16, kv, seed=20, mask_words=2)
    want, tol = b.reference()
    d = Dev(b)
    d.n[1] = 3            # fewer keys than rows
    d.n[2] = 16 * b.tables.shape[1] + 1  # beyond the table
    d.out.fill_(7.0)
    got = d.run(max_q=32)  # sequence 3 has more nodes than that
    assert pkv.pkv_device_errors() == 4
    got = got.cpu().double().numpy()
    assert (got[5:52] == 7.0).all()
    for a, e in ((0, 5), (52, 54)):
        assert np.abs(got[a:e] - want[a:e]).max() <= tol
    # a page out of range adds nothing: as if its keys were masked
    d = Dev(b)
    d.bt[0, 3], d.bt[4, 1] = b.nb, -1
    got = d.run().cpu().double().numpy()
    assert pkv.pkv_device_errors() == 2
    for s, lost in ((0, 3), (4, 1)):
        k, v = b.rows(s)
        keep = np.ones(b.n[s], bool)
        keep[16 * lost:16 * lost + 16] = False
        a = b.cu[s]
        ref, _ = tree_attention(b.q[a:a + b.q_lens[s]].double().numpy(), k[keep], v[keep], b.mask[a:a + b.q_lens[s]], b.scale)
        assert np.abs(got[a:a + b.q_lens[s]] - ref).max() <= tol


def test_rows_behind_the_last_sequence_stay():
    b = Batch([300, 20], [8, 5], 8, 2, 128, 16, "bf16", seed=21)
    d = Dev(b)
    want = d.run().clone()
    more = lambda t: torch.cat([t, t[:3]])  # noqa: E731
    out = torch.full((b.T + 3, 8, 128), 5.0, device="cuda")
    d.mask = more(d.mask)
    d.run(q=more(d.q), out=out)
    assert torch.equal(out[:b.T], want) and (out[b.T:] == 5.0).all()


def test_empty_calls():
    b = Batch([], [], 8, 2, 128, 16, "bf16", seed=1)
    d = Dev(b)
    d.run()
    b = Batch([20, 9], [0, 0], 8, 2, 128, 16, "bf16", seed=1)
    Dev(b).run()
    assert pkv.pkv_device_errors() == 0


def test_a_short_workspace_is_refused():
    b = Batch([3000], [8], 8, 2, 128, 16, "bf16", seed=22)
    d = Dev(b)
    need = pkv.pkv_tree_attention_workspace_size(d.q, d.bt, d.kc, b.max_q)
    if need:
        with pytest.raises(pkv.PkvError) as e:
            d.run(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 3
    full = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    d.run(workspace=full[:need])
    assert (full[need:] == 171).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_repeats_graphs_and_streams(kv):
    b = Batch([1800, 60, 700], [12, 3, 30], 8, 2, 128, 16, kv, seed=23)
    d = Dev(b)
    want = d.run().clone()
    ws = torch.empty(pkv.pkv_tree_attention_workspace_size(d.q, d.bt, d.kc, b.max_q), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        assert torch.equal(d.run(workspace=ws), want)
    outs = [torch.zeros_like(want) for _ in range(2)]
    graphs = []
    for o in outs:  # two graphs over one workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.run(workspace=ws, out=o)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    sides = [torch.cuda.Stream() for _ in range(3)]
    res = []
    torch.cuda.synchronize()
    for _ in range(5):  # calls at once, each with a workspace of its own
        for s in sides:
            with torch.cuda.stream(s):
                res.append(d.run(out=torch.empty_like(want)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in res)
    # the graph reads new lengths: one key fewer for every sequence changes its rows, as an eager call does
    d.n.sub_(1)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], d.run())
    assert pkv.pkv_device_errors() == 0


def test_a_chain_equals_causal_attention():
    """A chain of drafted tokens is an ordinary prefill chunk."""
    parents = [i - 1 for q in (8, 40) for i in range(q)]
    b = Batch([300, 700], [8, 40], 8, 2, 128, 16, "bf16", seed=24, parents=parents)
    d = compare(b)
    out = torch.empty_like(d.out)
    pkv.pkv_attention(d.q, d.cu, d.n, d.bt, d.kc, d.vc, b.scale, out, max_q_len=40)
    assert (out - d.out).abs().max() <= 2 * b.reference()[1]


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D,Hkv,bs", [(128, 8, 16), (64, 3, 12), (8, 1, 1), (40, 5, 7)])
def test_commit(kv, D, Hkv, bs):
    rng = np.random.default_rng(D)
    q_lens = [16, 1, 40, 7, 300, 5]
    b = Batch([100, 0, 33, 15, 2, 9], q_lens, Hkv, Hkv, D, bs, kv, seed=D)
    lens = [5, 1, 12, 7, 290, 0]
    acc = np.full((6, 300), -77, np.int32)
    for s, m in enumerate(lens):
        acc[s, :m] = np.sort(rng.permutation(q_lens[s])[:m])
    d = Dev(b)
    new = pkv.pkv_tree_commit(torch.from_numpy(acc).cuda()[:, :299 + 1], torch.tensor(lens, dtype=torch.int32).cuda(), d.cu,
                              d.n, d.bt, d.kc, d.vc)
    assert pkv.pkv_device_errors() == 0
    assert new.tolist() == [c + m for c, m in zip(b.ctx, lens)]
    for cache, got in ((b.kc, d.kc), (b.vc, d.vc)):
        want = cache.clone()
        for s, m in enumerate(lens):
            sl = b.slots(s)
            for i in range(m):  # ascending, one row at a time
                flat = want.view(torch.uint8).view(b.nb * bs, -1)
                flat[int(sl[b.ctx[s] + i])] = flat[int(sl[b.ctx[s] + acc[s, i]])]
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


def test_commit_refuses_inconsistent_paths():
    b = Batch([20] * 8, [6] * 8, 2, 2, 64, 16, "bf16", seed=3)
    d = Dev(b)
    acc = torch.tensor([[0, 2, 4], [2, 1, 3], [1, 1, 2], [0, 5, 6], [-1, 2, 3], [0, 1, 2], [1, 3, 5], [1, 2, 5]], dtype=torch.int32)
    lens = torch.tensor([3, 3, 3, 3, 3, 4, 3, -1], dtype=torch.int32)
    d.bt[6, 1] = b.nb  # the block that holds the drafted rows of sequence 6
    new = pkv.pkv_tree_commit(acc.cuda(), lens.cuda(), d.cu, d.n, d.bt, d.kc, d.vc)
    assert pkv.pkv_device_errors() == 6
    assert new.tolist() == [23, 26, 26, 26, 26, 26, 26, 26]
    want = b.kc.clone()
    sl = b.slots(0)
    for i, a in enumerate([0, 2, 4]):
        want.view(-1, 2, 64)[int(sl[20 + i])] = want.view(-1, 2, 64)[int(sl[20 + a])]
    assert torch.equal(d.kc.cpu(), want)


# ---------------------------------------------------------------- a whole step
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_speculative_step(kv, captured):
    """Mask, slots, rotary append, attention, commit, and the next decode over
    the kept rows, eagerly and from a graph, against a plain 64-bit step."""
    from tests.spec_ref import frequencies, rotate, attention_tolerance
    rng = np.random.default_rng(7)
    Hq, Hkv, D, bs = 8, 2, 128, 16
    b = Batch([500, 0, 37], [12, 5, 9], Hq, Hkv, D, bs, kv, seed=31)
    gen = torch.Generator().manual_seed(8)
    qkv = torch.randn((b.T, Hq + 2 * Hkv, D), generator=gen).bfloat16()
    paths, lens = np.zeros((3, 4), np.int32), [4, 2, 3]
    for s, m in enumerate(lens):
        paths[s, :m] = np.sort(rng.permutation(b.q_lens[s])[:m])
    d = Dev(b)
    rope = pkv.pkv_rope_init(D, 10000.0)
    dev, acc, al = qkv.cuda(), torch.from_numpy(paths).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    kc0, vc0 = d.kc.clone(), d.vc.clone()
    mask = torch.empty((b.T, 1), dtype=torch.int32, device="cuda")
    pos, new_n = torch.empty(b.T, dtype=torch.int32, device="cuda"), torch.empty_like(d.n)
    slots, q2 = torch.empty(b.T, dtype=torch.int32, device="cuda"), torch.empty((b.T, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.pkv_tree_attention_workspace_size(q2, d.bt, d.kc, 12), dtype=torch.uint8, device="cuda")

    def step():
        pkv.pkv_tree_mask(d.parents, d.cu, d.n, 12, tree_mask=mask, positions=pos)
        pkv.pkv_slot_mapping(d.cu, d.n, d.bt, bs, out=slots)
        pkv.pkv_rope_append(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], pos, slots, rope, d.kc, d.vc, q_out=q2,
                            k_scale=b.k_scale, v_scale=b.v_scale)
        pkv.pkv_tree_attention(q2, d.cu, d.n, d.bt, d.kc, d.vc, mask, b.scale, d.out, b.k_scale, b.v_scale, 12, ws)
        pkv.pkv_tree_commit(acc, al, d.cu, d.n, d.bt, d.kc, d.vc, new_n)

    step()
    if captured:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        d.kc.copy_(kc0)
        d.vc.copy_(vc0)
        d.out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert pkv.pkv_device_errors() == 0
    # the plain step, on what the cache holds after the append (its own rounding is the append test's)
    f, amp = frequencies(D, 10000.0)
    k_new = rotate(qkv.double().numpy()[:, Hq:Hq + Hkv], b.pos, f, amp, D, False)
    new_lens = new_n.tolist()
    assert new_lens == [c + m for c, m in zip(b.ctx, lens)]
    got, q_rot = d.out.cpu().double().numpy(), q2.cpu().double().numpy()
    step_tol = 2.0 ** -7 * np.abs(k_new).max() if kv == "bf16" else 2.0 ** -3 * np.abs(k_new).max() + b.k_scale
    b.kc, b.vc = kc0.cpu(), vc0.cpu()
    for s in range(3):
        a, e, sl = b.cu[s], b.cu[s + 1], torch.from_numpy(b.slots(s))
        # the rows of the tree as the append stored them
        kk, vv = kc0.clone(), vc0.clone()
        pkv.pkv_append(torch.from_numpy(k_new[a:e]).bfloat16().cuda(), dev[a:e, Hq + Hkv:], slots[a:e], kk, vv, b.k_scale,
                       b.v_scale)
        b.kc, b.vc = kk.cpu(), vv.cpu()
        k, v = b.rows(s)
        want, top = tree_attention(q_rot[a:e], k, v, b.mask[a:e], b.scale)
        # two bf16 or e4m3 roundings of k may differ by a step: the score by |q|.|dk|, far below step_tol * sum|q|
        tol = attention_tolerance(np.abs(v).max(), top, b.n[s], kv) + 2 * np.abs(v).max() * np.expm1(
            min(5.0, b.scale * np.abs(q_rot[a:e]).sum(-1).max() * step_tol))
        assert np.abs(got[a:e] - want).max() <= tol
        # the kept rows are the accepted nodes', in order
        kept = d.kc.cpu().double().view(-1, Hkv, D)[sl[b.ctx[s]:b.ctx[s] + lens[s]]].numpy() * b.k_scale
        assert np.abs(kept - k_new[a:e][paths[s, :lens[s]]]).max() <= step_tol
        same = d.vc.cpu().view(torch.uint8).view(b.nb * bs, -1)[sl[b.ctx[s]:b.ctx[s] + lens[s]]]
        assert torch.equal(same, vv.cpu().view(torch.uint8).view(b.nb * bs, -1)[sl[b.ctx[s]:][torch.from_numpy(paths[s, :lens[s]]).long()]])
    # and the library's own decode goes on from there
    out = torch.empty((3, Hq, D), device="cuda")
    cu1 = torch.arange(4, dtype=torch.int32, device="cuda")
    pkv.pkv_attention(q2[:3].contiguous(), cu1, new_n, d.bt, d.kc, d.vc, b.scale, out, b.k_scale, b.v_scale, max_q_len=1)
    tree = torch.empty_like(out)
    pkv.pkv_tree_attention(q2[:3].contiguous(), cu1, new_n, d.bt, d.kc, d.vc, torch.ones((3, 1), dtype=torch.int32, device="cuda"),
                           b.scale, tree, b.k_scale, b.v_scale, 1)
    b.kc, b.vc = d.kc.cpu(), d.vc.cpu()
    vmax = float(max(np.abs(b.rows(s)[1]).max() for s in range(3)))
    top = float(b.scale * np.abs(q_rot[:3]).sum(-1).max() * 6)
    assert (out - tree).abs().max() <= 2 * attention_tolerance(vmax, top, 512, kv)
    assert pkv.pkv_device_errors() == 0
