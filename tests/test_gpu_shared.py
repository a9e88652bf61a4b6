"""Attention of requests that share prefixes against plain 64-bit references,
where it can go wrong: groups of one and of many, rows of one and of many
tiles, prefixes that end inside a tile, values that must not leak, bad groups,
lengths and pages, strides, streams and graphs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.share_ref import SharedBatch
from tests.test_gpu_tree import poison

pytestmark = pytest.mark.gpu


class Dev:
    def __init__(self, b, out_dtype=torch.float32):
        c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.b = b
        self.q, self.kc, self.vc = b.q.cuda(), b.kc.cuda(), b.vc.cuda()
        self.cu, self.n, self.bt = c(b.cu), c(np.array(b.n, np.int32)), c(b.tables)
        self.groups = torch.tensor(b.groups, dtype=torch.int32, device="cuda").view(-1, 3)
        self.out = torch.full((b.T, b.Hq, b.D), 7.0, dtype=out_dtype, device="cuda")

    def run(self, max_q=None, max_group=None, **kw):
        b = self.b
        return pkv.pkv_shared_attention(kw.pop("q", self.q), self.cu, self.n, self.bt, self.groups, self.kc, self.vc,
                                        kw.pop("scale", b.scale), kw.pop("out", self.out), k_scale=b.k_scale, v_scale=b.v_scale,
                                        max_q_len=b.max_q if max_q is None else max_q,
                                        max_group_len=b.max_group if max_group is None else max_group, **kw)


def close(b, got, rows=None):
    want, tol = b.reference()
    got = got.cpu().double().numpy()
    if rows is not None:
        want, got = want[rows], got[rows]
    both = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), both)
    err = np.abs(got[both] - want[both])
    assert err.size == 0 or err.max() <= tol, f"max err {err.max():.3e}, tolerance {tol:.3e}"


def compare(b, flags=0, **kw):
    d = Dev(b)
    d.run(**kw)
    assert pkv.pkv_device_errors() == flags
    close(b, d.out)
    return d


SHAPES = [  # groups, own context, new tokens, Hq, Hkv, D, bs
    ([(4, 1024)], [16, 100, 0, 77], [1] * 4, 32, 8, 128, 16),
    ([(1, 64)], [5], [1], 4, 4, 64, 16),
    ([(2, 16), (1, 0), (3, 256)], [0, 1, 300, 127, 128, 129], [1, 2, 1, 3, 1, 1], 8, 2, 128, 16),
    ([(9, 300), (2, 12), (1, 24), (1, 0)], [0] * 6 + [11, 250, 3, 400, 1, 0, 0], [1, 2, 3, 4, 5, 6, 7, 1, 1, 2, 1, 3, 1], 15, 3, 64, 12),
    ([(40, 512)], list(range(40)), [1] * 40, 16, 4, 128, 16),         # 160 rows: 128-row tiles, one of them odd
    ([(5, 128), (3, 128)], [60] * 8, [30, 1, 64, 0, 33, 70, 2, 9], 8, 2, 64, 32),  # wide own rows
    ([(17, 1)], [3] * 17, [1] * 17, 7, 1, 128, 1),
    ([(3, 2100)], [500, 0, 1300], [2, 2, 1], 6, 6, 128, 7),
    ([(2, 127), (2, 127), (2, 129)], [0, 1, 127, 0, 1, 0], [1] * 6, 2, 1, 64, 1),
    ([(3, 4992), (2, 64)], [5000, 3, 100, 7000, 1], [1, 3, 1, 1, 2], 4, 2, 128, 16),
    ([(6, 64)], [2] * 6, [1, 0, 2, 0, 0, 1], 160, 2, 64, 16),         # many heads for a KV head
    ([(2, 0), (2, 0)], [90, 0, 2, 130], [4, 1, 1, 130], 2, 2, 128, 4),  # nothing shared
    ([(70, 192)], [9] * 70, [1] * 70, 1, 1, 64, 64),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shared_attention(shape, kv):
    b = SharedBatch(*SHAPES[shape], kv=kv, seed=300 + shape)
    compare(b)
    compare(b, max_q=0, max_group=0)  # bounds unknown: other tiles


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_f32(D):
    compare(SharedBatch([(3, 48), (1, 0), (2, 16)], [7, 0, 30, 64, 5, 1], [1, 3, 0, 2, 1, 4], 6, 2, D, 16, "f32", seed=D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_long_prefix_and_long_requests(kv):
    compare(SharedBatch([(3, 40000)], [9000, 1, 20000], [1, 2, 1], 4, 2, 64, 16, kv, seed=3))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_several_items_for_each_cta(kv):
    """More groups and requests than SMs: every role goes round its rings."""
    g = [(4, 256)] * 60
    b = SharedBatch(g, [17 * s % 400 for s in range(240)], [1] * 240, 8, 4, 64, 16, kv, seed=8)
    d = compare(b)
    again = d.run(out=torch.empty_like(d.out))
    assert torch.equal(d.out, again)  # bit for bit


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bf16_output_is_the_rounded_f32_output(kv):
    b = SharedBatch([(3, 256), (1, 0)], [700, 33, 0, 50], [1, 4, 2, 1], 8, 2, 128, 16, kv, seed=5)
    f = Dev(b).run().clone()
    h = Dev(b, torch.bfloat16).run()
    assert torch.equal(h, f.to(torch.bfloat16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name,shape", [
    ("many requests", ([(25, 16)] * 60, [s % 20 for s in range(1500)], [1] * 1500, 2, 1, 64, 16)),
    ("many rows behind a prefix", ([(2, 64), (40, 96)], [0, 90] + [5] * 40, [2100, 2300] + [1] * 40, 2, 1, 64, 32)),
    ("rows enough for tiles of their own", ([(5, 512)], [0, 7, 100, 300, 64], [130, 64, 200, 90, 128], 8, 4, 64, 16)),
    ("more KV heads than SMs", ([(3, 32)], [4, 40, 0], [1, 2, 1], 320, 160, 64, 16)),
    ("one long request among short ones", ([(30, 128)], [1] * 29 + [30000], [1] * 30, 2, 2, 64, 16)),
])
def test_large_and_uneven_batches(name, shape, kv):
    compare(SharedBatch(*shape, kv=kv, seed=len(name)))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,q", [(1, 1), (4, 2), (5, 3), (8, 4), (8, 8), (8, 9)])
def test_groups_whose_rows_need_no_larger_tile_than_their_requests(G, q, kv):
    # pairs of requests of 9 to 16, 17 to 32, .. rows and some alone, in more than one set
    # of 32 requests; every ninth has no rows, every seventh no keys of its own but the new
    r = np.random.default_rng(900 + 10 * G + q)
    groups = [(2 if i % 4 else 1, int(r.integers(0, 9)) * 48) for i in range(42)]
    B = sum(g for g, _ in groups)
    own = [0 if i % 7 == 3 else int(r.integers(0, 700)) for i in range(B)]
    new = [0 if i % 9 == 5 else 1 + (i * 5) % q for i in range(B)]
    b = SharedBatch(groups, own, new, 2 * G, 2, 64 if q & 1 else 128, 48, kv=kv, seed=900 + 10 * G + q)
    d = compare(b)
    first = d.out.clone()
    compare(b, max_group=max(new) * B)  # other tiles for the groups
    d.out.fill_(7.0)
    d.run()
    assert torch.equal(first, d.out)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_blocks_beyond_two_billion_elements(kv):
    b = SharedBatch([(3, 64), (1, 0)], [40, 3, 170, 90], [1, 2, 1, 1], 8, 2, 128, 16, kv, seed=47)
    blocks = (1 << 31) // (16 * 2 * 128) + 5000  # an element's number passes 31 bits
    d = Dev(b)
    old = [d.kc, d.vc]
    d.kc, d.vc = (torch.empty((blocks, 16, 2, 128), dtype=x.dtype, device="cuda") for x in old)
    for x, y in zip(old, (d.kc, d.vc)):
        y[-b.nb:].view(torch.uint8).copy_(x.view(torch.uint8))
    d.bt = torch.where(d.bt >= 0, d.bt + (blocks - b.nb), d.bt)
    d.run()
    assert pkv.pkv_device_errors() == 0
    close(b, d.out)


def test_requests_without_a_prefix_are_pkv_attention():
    b = SharedBatch([(1, 0)] * 5, [300, 0, 17, 1000, 64], [1, 1, 1, 1, 1], 8, 2, 128, 16, "bf16", seed=2)
    d = compare(b)
    want = pkv.pkv_attention(d.q, d.cu, d.n, d.bt, d.kc, d.vc, b.scale, torch.empty_like(d.out), max_q_len=1)
    assert (want - d.out).abs().max() <= 2 * b.reference()[1]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_block_size_and_placement_do_not_matter(kv):
    """The same keys in blocks of 16 and of 64, elsewhere in the pool: the same bits."""
    shape = ([(5, 512), (2, 64)], [100, 3, 0, 70, 9, 200, 1], [1, 2, 1, 3, 1, 1, 1], 8, 2, 128)
    a, b = SharedBatch(*shape, 16, kv, seed=4), SharedBatch(*shape, 64, kv, seed=6)
    width = 1024
    for x in (a, b):  # the tables' width is among the shapes that choose the cut
        t = np.full((x.B, width // x.bs), -1, np.int32)
        t[:, :x.tables.shape[1]] = x.tables
        x.tables = t
    b.q = a.q
    bits = torch.int16 if kv == "bf16" else torch.uint8
    for s in range(a.B):
        for x, y in ((a.kc, b.kc), (a.vc, b.vc)):
            y.view(bits).view(-1, 2, 128)[torch.from_numpy(b.slots(s))] = x.view(bits).view(-1, 2, 128)[torch.from_numpy(a.slots(s))]
    assert torch.equal(Dev(a).run(), Dev(b).run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_a_row_does_not_depend_on_the_other_requests(kv):
    b = SharedBatch([(4, 128), (2, 64)], [100, 3, 0, 70, 9, 200], [1, 2, 1, 3, 1, 1], 8, 2, 64, 16, kv, seed=14)
    d = Dev(b)
    first = d.run().clone()
    mine = slice(int(b.cu[2]), int(b.cu[3]))
    d.q = torch.where((torch.arange(b.T, device="cuda") == mine.start)[:, None, None], d.q, -d.q)
    d.n[5] -= 90
    assert torch.equal(d.run()[mine], first[mine])


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_unseen_values_do_not_leak(kv):
    b = SharedBatch([(3, 64), (1, 0), (40, 32)], [150, 0, 64, 20] + [1] * 40, [6, 9, 3, 40] + [1] * 40, 8, 2, 64, 16, kv, seed=13)
    bad = [float("nan")] + ([] if kv == "e4m3" else [float("inf"), -float("inf")])
    used = torch.zeros(b.nb * b.bs, dtype=torch.bool)
    for s in range(b.B):
        used[torch.from_numpy(b.slots(s))] = True
    for c in (b.kc, b.vc):  # outside the requests
        poison(c, ~used, bad[0])
    # new tokens that hold poison: only rows behind them may show it
    for s, at in ((0, 3), (1, 0), (3, 39)):
        slot = int(b.slots(s)[b.ctx[s] + at])
        if s == 1:
            poison(b.kc, slot, bad[0])
        else:
            poison(b.vc, slot, bad[s % len(bad)])
    d = Dev(b)
    d.run()
    assert pkv.pkv_device_errors() == 0
    got = d.out.cpu()
    rows = lambda s, a, e: slice(int(b.cu[s]) + a, int(b.cu[s]) + e)  # noqa: E731
    clean = np.ones(b.T, bool)
    for s, at in ((0, 3), (1, 0), (3, 39)):
        clean[rows(s, at, b.q_lens[s])] = False
        assert not torch.isfinite(got[rows(s, at, b.q_lens[s])]).any()
    assert torch.isfinite(got[torch.from_numpy(clean)]).all()
    close(b, got, np.nonzero(clean)[0])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_scales(kv, scale):
    b = SharedBatch([(30, 128)], [9] * 30, [1] * 30, 8, 2, 64, 16, kv, seed=21)
    b.scale = scale
    compare(b)


# ---------------------------------------------------------------- what is refused on the device
GROUPS = {  # group of requests 0 .. 3, then 4, then 5 .. 6
    "prefix beyond the context": lambda g: g[:4, 2].fill_(1 << 20),
    "prefix inside a block": lambda g: g[:4, 2].fill_(40),
    "negative prefix": lambda g: g[:4, 2].fill_(-16),
    "first behind the request": lambda g: g[:4, 0].fill_(4),
    "first below zero": lambda g: g[:4, 0].fill_(-1),
    "end behind the batch": lambda g: g[:4, 1].fill_(9),
    "end before the request": lambda g: g[:4, 1].fill_(0),
    "first of another group": lambda g: g[:4, 0].fill_(0) + g[0, 0].fill_(3),
    "first with another prefix": lambda g: g[0, 2].fill_(16),
    "first without a prefix": lambda g: g[0, 2].fill_(0),
    "huge": lambda g: g[:4].fill_(2147483632),
    "smallest": lambda g: g[:4].fill_(-2147483648),
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("name", list(GROUPS))
def test_bad_groups_are_recorded(name, kv):
    b = SharedBatch([(4, 64), (1, 0), (2, 32)], [40, 3, 17, 1, 30, 8, 1], [1, 2, 1, 1, 3, 1, 1], 4, 2, 64, 16, kv, seed=31)
    d = Dev(b)
    GROUPS[name](d.groups)
    d.run()
    assert pkv.pkv_device_errors() == 4
    got = d.out.cpu()
    first = int(b.cu[4])
    close(b, got, slice(first, None))
    for s in range(4):  # left as they were, or (a request whose own numbers hold) right
        rows = slice(int(b.cu[s]), int(b.cu[s + 1]))
        if not (got[rows] == 7.0).all():
            assert name in ("first with another prefix", "first without a prefix") and s == 0
            close(b, got, rows)


def test_a_context_shorter_than_the_prefix_is_its_own_matter():
    b = SharedBatch([(3, 64)], [40, 3, 17], [1, 2, 1], 4, 2, 64, 16, "bf16", seed=32)
    for s in range(3):  # the first one's table is still read for the others
        d = Dev(b)
        d.n[s] = 60
        d.run()
        assert pkv.pkv_device_errors() == 4
        for r in range(3):
            rows = slice(int(b.cu[r]), int(b.cu[r + 1]))
            if r == s:
                assert (d.out[rows] == 7.0).all()
            else:
                close(b, d.out, rows)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_more_rows_than_the_bounds(kv):
    b = SharedBatch([(2, 32), (3, 16)], [5, 6, 7, 8, 9], [1, 1, 2, 3, 1], 4, 2, 64, 16, kv, seed=33)
    d = Dev(b)
    d.run(max_q=2)
    assert pkv.pkv_device_errors() == 4
    assert (d.out[int(b.cu[3]):int(b.cu[4])] == 7.0).all()
    close(b, d.out, [0, 1, 2, 3, 7])
    d = Dev(b)
    d.run(max_q=3, max_group=5)
    assert pkv.pkv_device_errors() == 4
    assert (d.out[2:] == 7.0).all()
    close(b, d.out, [0, 1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_bad_lengths(kv):
    b = SharedBatch([(2, 32), (1, 0), (1, 0)], [5, 6, 7, 8], [1, 1, 2, 3], 4, 2, 64, 16, kv, seed=34)
    for change in (lambda d: d.n.__setitem__(2, 1), lambda d: d.n.__setitem__(2, 1 << 30), lambda d: d.n.__setitem__(2, -5)):
        d = Dev(b)
        change(d)
        d.run()
        assert pkv.pkv_device_errors() == 4
        assert (d.out[2:4] == 7.0).all()
        close(b, d.out, [0, 1, 4, 5, 6])
    for at, value in ((1, 5), (1, -1), (4, 100), (0, -2), (2, 1 << 30)):
        d = Dev(b)
        d.cu[at] = value
        d.run()
        assert pkv.pkv_device_errors() == 4


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("bs", [16, 12, 1])
def test_bad_pages_add_nothing(kv, bs):
    b = SharedBatch([(3, 10 * bs), (1, 0)], [70, 3, 17, 200], [1, 2, 1, 3], 4, 2, 64, bs, kv, seed=35)
    d = Dev(b)
    where = {0: [2], 1: [2], 2: [2, 10], 3: [0, 1]}  # blocks: one of the prefix, some of their own
    for s, blocks in where.items():
        for j in blocks:
            d.bt[s, j] = -3 if j % 2 else b.nb
    d.run()
    assert pkv.pkv_device_errors() == 2
    for s, blocks in where.items():  # the reference: those keys are hidden by a mask of their own
        k, v = b.rows(s)
        keep = np.ones(b.n[s], bool)
        for j in blocks:
            keep[j * bs:(j + 1) * bs] = False
        for i in range(b.q_lens[s]):
            see = keep & (np.arange(b.n[s]) <= b.ctx[s] + i)
            t = int(b.cu[s]) + i
            for h in range(b.Hq):
                x = b.scale * (k[see, h // 2] @ b.q[t, h].double().numpy())
                w = np.exp(x - x.max())
                ref = w @ v[see, h // 2] / w.sum()
                assert np.abs(ref - d.out[t, h].cpu().double().numpy()).max() <= b.reference()[1]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_no_page_at_all_gives_zeros(kv):
    b = SharedBatch([(2, 32)], [5, 6], [1, 2], 4, 2, 64, 16, kv, seed=36)
    d = Dev(b)
    d.bt.fill_(-1)
    d.run()
    assert pkv.pkv_device_errors() == 2
    assert (d.out == 0).all()


# ---------------------------------------------------------------- how it is called
def test_strides_and_rows_behind_the_last():
    b = SharedBatch([(3, 64), (1, 0)], [40, 3, 17, 9], [1, 2, 1, 3], 8, 2, 64, 16, "bf16", seed=41)
    d = Dev(b)
    fused = torch.full((b.T + 4, 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:b.T, :8] = d.q
    out = torch.full((b.T + 4, 10, 72), 7.0, device="cuda")
    bt = torch.full((b.B, b.tables.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    bt[:, :b.tables.shape[1]] = d.bt
    d.bt = bt[:, :b.tables.shape[1]]
    d.run(q=fused[:, :8], out=out[:, 1:9, :64])
    assert pkv.pkv_device_errors() == 0
    close(b, out[:b.T, 1:9, :64])
    assert (out[b.T:] == 7.0).all() and (out[:, 0] == 7.0).all() and (out[:, 9] == 7.0).all() and (out[:, :, 64:] == 7.0).all()


def test_nothing_to_do():
    b = SharedBatch([(2, 32)], [5, 6], [0, 0], 4, 2, 64, 16, "bf16", seed=42)
    d = Dev(b)
    d.run()
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, 4, 64), 7.0, device="cuda")
    d.run(q=q, out=out)
    assert pkv.pkv_device_errors() == 0 and (out == 7.0).all()


def test_another_stream_and_two_calls_at_once():
    shape = ([(8, 512)], [50] * 8, [1] * 8, 8, 2, 128, 16)
    a, b = Dev(SharedBatch(*shape, "bf16", seed=43)), Dev(SharedBatch(*shape, "e4m3", seed=44))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    torch.cuda.synchronize()
    assert pkv.pkv_device_errors() == 0
    close(a.b, a.out)
    close(b.b, b.out)


def test_graphs_that_share_a_workspace_follow_their_inputs():
    b = SharedBatch([(6, 256), (2, 64)], [50, 3, 0, 200, 17, 1, 90, 4], [1] * 8, 8, 2, 64, 16, "bf16", seed=45)
    d, e = Dev(b), Dev(b)
    d.run()  # one-time set-up
    ws = torch.empty(pkv.pkv_shared_attention_workspace_size(d.q, d.bt, d.kc, 1, 8), dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (d, e):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(max_group=8, workspace=ws)
        graphs.append(g)
    d.out.fill_(7.0)
    e.q.neg_()
    for g in graphs + graphs:
        g.replay()
    assert pkv.pkv_device_errors() == 0
    close(b, d.out)
    want = e.run(max_group=8, out=torch.empty_like(e.out))
    assert torch.equal(e.out, want)
    # other groups and lengths, replayed: nothing of the first ones is kept
    d.groups.copy_(pkv.pkv_shared_prefixes(d.cu, d.n, d.bt, 16, min_tokens=100))
    d.out.fill_(7.0)
    graphs[0].replay()
    close(b, d.out)
    assert d.groups.tolist()[7] == [7, 8, 0]
    d.groups.zero_()
    d.out.fill_(7.0)
    graphs[0].replay()
    assert pkv.pkv_device_errors() == 0
    close(b, d.out)


def test_workspace_that_is_too_small():
    b = SharedBatch([(2, 32)], [5, 6], [1, 1], 4, 2, 64, 16, "bf16", seed=46)
    d = Dev(b)
    n = pkv.pkv_shared_attention_workspace_size(d.q, d.bt, d.kc, 1, 2)
    with pytest.raises(pkv.PkvError) as e:
        d.run(workspace=torch.empty(n - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(pkv.PkvError):
        d.run(workspace=torch.empty(n + 16, dtype=torch.uint8, device="cuda")[16:])
    assert (d.out == 7.0).all()
