"""pkv_step_tables and pkv_shared_prefixes on the GPU against the plain
references: whole numbers, equal bit for bit."""
import random

import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests import share_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Step:
    """Device state of a step, and the reference's answer."""

    def __init__(self, old, new, bs, tables, free, count, T, shared=None, i64=False, positions=True, stride=0, in_place=True):
        B = len(old)
        sh = shared if shared is not None else [0] * B
        self.want = share_ref.step_tables(old, new, sh, bs, tables, free, count, T)
        W = len(tables[0]) if B else 1
        self.whole = torch.full((B, W + stride), -77, dtype=torch.int32, device=DEV)
        self.bt = self.whole[:, :W]
        if B:
            self.bt.copy_(i32(tables))
        self.free, self.count = i32(free), i32([count])
        self.left = self.count if in_place else i32([-5])
        self.cu = torch.full((B + 1,), -9, dtype=torch.int32, device=DEV)
        self.slots = torch.full((T,), -9, dtype=torch.int64 if i64 else torch.int32, device=DEV)
        self.pos = torch.full((T,), -9, dtype=torch.int32, device=DEV) if positions else None
        self.args = (i32(old), i32(new), self.bt, bs, self.free, self.count, self.cu, self.slots)
        self.kw = dict(shared_blocks=i32(shared) if shared is not None else None, positions=self.pos, new_free_count=None if in_place else self.left)

    def run(self):
        pkv.pkv_step_tables(*self.args, **self.kw)

    def check(self, flags=None):
        tables, free, count, cu, slots, positions, bits = self.want
        assert pkv.pkv_device_errors() == (bits if flags is None else flags)
        assert self.bt.tolist() == tables
        assert (self.whole[:, self.bt.shape[1]:] == -77).all()
        assert self.free.tolist() == free and self.left.tolist() == [count]
        assert self.cu.tolist() == cu and self.slots.tolist() == slots
        if self.pos is not None:
            assert self.pos.tolist() == positions


def step(seed, B, bs, old_hi, grow, T_pad=0, shared=False, spare=5, **kw):
    r = random.Random(seed)
    old, new, sh = [], [], []
    for _ in range(B):
        s = r.randint(0, 4) if shared and r.random() < 0.5 else 0
        a = s * bs + r.randint(0, old_hi)
        u = r.random()
        b = 0 if u < 0.15 else max(0, a - r.randint(0, 9)) if u < 0.3 else a if u < 0.35 else a + r.randint(1, grow)
        old.append(a)
        new.append(b)
        sh.append(s)
    W = max(-(-max(a, b) // bs) for a, b in zip(old, new)) + 2
    ids = r.sample(range(10 * B * W + 1000), B * W + 1000)
    tables = [[ids.pop() if j < -(-a // bs) else -1 for j in range(W)] for a in old]
    taken = sum(max(0, -(-b // bs) + -a // bs) for a, b in zip(old, new))
    count = taken + spare
    free = [ids.pop() if k < count and ids else -1 for k in range(count + B * W)]
    T = sum(max(0, b - a) for a, b in zip(old, new)) + T_pad
    return Step(old, new, bs, tables, free, count, T, sh if shared else None, **kw)


@pytest.mark.parametrize("bs", [1, 3, 12, 16, 64])
@pytest.mark.parametrize("B,old_hi,grow", [(1, 50, 4), (7, 100, 1), (64, 400, 8), (33, 300, 200), (300, 60, 30)])
def test_steps(bs, B, old_hi, grow):
    st = step(B + bs, B, bs, old_hi, grow)
    st.run()
    st.check()
    st = step(B + bs + 1, B, bs, old_hi, grow, T_pad=5, shared=True, i64=True, stride=3, in_place=False)
    st.run()
    st.check()


@pytest.mark.parametrize("B", [1023, 1024, 1025, 3000, 8192])
def test_many_requests(B):
    st = step(B, B, 16, 40, 3, shared=True)
    st.run()
    st.check()


@pytest.mark.parametrize("T", [1, 1024, 1025, 2049, 4097, 9000, 40000])
def test_long_prompts_take_one_or_more_ctas(T):
    r = random.Random(T)
    bs, n = 16, -(-T // 16) + 1
    ids = r.sample(range(5 * n + 50), n + 20)
    old, new = [5, 0, 40], [5 + T, 0, 0]
    tables = [[ids.pop()] + [-1] * n, [-1] * (n + 1), [ids.pop(), ids.pop(), ids.pop()] + [-1] * (n - 2)]
    free = ids + [-1] * 4
    st = Step(old, new, bs, tables, free, len(ids), T)
    st.run()
    st.check()


def test_nothing_to_do():
    st = Step([], [], 16, [], [4, 3], 2, 6)
    st.run()
    st.check()
    st = Step([0, 17, 5], [0, 17, 5], 16, [[1, 2]] * 3, [4, 3], 2, 0, positions=False)
    st.run()
    st.check()


def test_what_is_given_back_is_taken_at_once():
    # the list is empty: request 0's blocks go to request 1, last first
    st = Step([48, 16], [0, 60], 16, [[10, 11, 12, -1], [20, -1, -1, -1]], [0, 0, 0], 0, 44)
    st.run()
    st.check()
    assert st.bt.tolist()[1] == [20, 12, 11, 10]


REFUSED = {
    "out of blocks": dict(old=[16, 3], new=[33, 60], count=3, T=80),
    "list too short": dict(old=[64, 3], new=[0, 4], count=6, F=8),
    "count below zero": dict(old=[16, 3], new=[17, 4], count=-1),
    "count beyond the list": dict(old=[16, 3], new=[17, 4], count=9, F=8),
    "more rows than slots": dict(old=[16, 3], new=[17, 8], count=4, T=5),
    "no slots": dict(old=[16, 3], new=[17, 3], count=4, T=0),
    "beyond the table": dict(old=[16, 3], new=[65, 4], count=8),
    "negative": dict(old=[-1, 3], new=[4, 4], count=8),
    "below zero": dict(old=[16, 3], new=[-2147483648, 4], count=8),
    "rows among shared blocks": dict(old=[16, 3], new=[17, 4], count=8, shared=[2, 0]),
    "shared beyond the table": dict(old=[16, 3], new=[0, 4], count=8, shared=[5, 0]),
    "shared below zero": dict(old=[16, 3], new=[0, 4], count=8, shared=[-1, 0]),
    "huge": dict(old=[0, 0], new=[2147483647, 2147483647], count=8),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_refused_steps(name):
    c = REFUSED[name]
    F = c.get("F", 12)
    T = c.get("T", 64)
    tables = [[1, 2, 3, 4], [5, 6, 7, 8]]
    st = Step(c["old"], c["new"], 16, tables, list(range(20, 20 + F)), c["count"], T, c.get("shared"))
    assert st.want[6] != 0
    st.run()
    st.check()


def test_a_negative_block_gives_no_slot():
    st = Step([3, 0], [5, 3], 4, [[-1, -1], [-1, -1]], [9, -4, 7], 2, 5)
    assert st.want[6] == 2
    st.run()
    st.check()
    # slots beyond int32 have no place in an int32 mapping
    st = Step([3, 0], [5, 3], 4, [[1 << 30, -1], [-1, -1]], [9, 4, 7], 3, 5)
    st.run()
    assert pkv.pkv_device_errors() == 1
    assert st.slots.tolist() == [-1, 28, 16, 17, 18]


def test_captured_and_replayed_steps_follow_the_lengths():
    """One graph, several steps: lengths, list and count are read when it runs."""
    B, bs, W = 6, 4, 8
    pkv.pkv_step_tables(*step(0, B, bs, 10, 2).args)  # one-time set-up outside the capture
    torch.cuda.synchronize()
    pkv.pkv_device_errors()
    old, new = i32([0] * B), i32([0] * B)
    bt, free, count = torch.full((B, W), -1, dtype=torch.int32, device=DEV), torch.randperm(64, device=DEV).to(torch.int32), i32([64])
    cu, slots = torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(64, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_step_tables(old, new, bt, bs, free, count, cu, slots)
        old.copy_(new)
    r = random.Random(4)
    tables, lst, n, a = bt.tolist(), free.tolist(), 64, [0] * B
    for _ in range(12):
        b = [0 if r.random() < 0.2 else min(30, x + r.randint(-4, 9)) if x else r.randint(0, 10) for x in a]
        b = [max(0, x) for x in b]
        tables, lst, n, wcu, wslots, _, flags = share_ref.step_tables(a, b, [0] * B, bs, tables, lst, n, 64)
        new.copy_(i32(b))
        g.replay()
        assert pkv.pkv_device_errors() == flags == 0
        assert (bt.tolist(), free.tolist(), count.tolist(), cu.tolist(), slots.tolist()) == (tables, lst, [n], wcu, wslots)
        a = b


def test_slots_equal_those_of_the_slot_mapping():
    st = step(9, 40, 16, 200, 30)
    st.run()
    want = pkv.pkv_slot_mapping(st.cu, torch.maximum(st.args[0], st.args[1]), st.bt, 16, T=st.slots.shape[0])
    assert torch.equal(st.slots, want)
    assert pkv.pkv_device_errors() == 0


# ---------------------------------------------------------------- shared prefixes
def batch(seed, B, bs, blocks, q_hi=3, drop=0.1, wide=0):
    """Requests in groups that share some blocks."""
    r = random.Random(seed)
    tables, n, cu, ids = [], [], [0], list(range(1, 1 << 16))
    r.shuffle(ids)
    prev = []
    for _ in range(B):
        own = r.randint(0, blocks)
        keep = r.choice([0, len(prev), len(prev) // 2, r.randint(0, len(prev))])
        row = prev[:keep] + [ids[r.randrange(len(ids))] for _ in range(own)]
        q = r.randint(0, q_hi)
        m = max(q, len(row) * bs - r.randint(0, bs - 1) if row else 0)
        row = row + [ids[r.randrange(len(ids))] for _ in range(-(-m // bs) - len(row))]
        if row and r.random() < drop:
            row[r.randrange(len(row))] = -1
        tables.append(row)
        n.append(m)
        cu.append(cu[-1] + q)
        prev = row[:-(-m // bs)]
    W = max(map(len, tables)) + 1 + wide
    return cu, n, [t + [-1] * (W - len(t)) for t in tables]


@pytest.mark.parametrize("bs", [1, 12, 16])
@pytest.mark.parametrize("B,blocks,least", [(1, 4, 1), (2, 3, 1), (9, 5, 16), (64, 8, 30), (300, 3, 1), (1500, 4, 20)])
def test_groups(bs, B, blocks, least):
    cu, n, tables = batch(B + bs, B, bs, blocks)
    want, flags = share_ref.shared_prefixes(cu, n, tables, bs, least)
    got = pkv.pkv_shared_prefixes(i32(cu), i32(n), i32(tables), bs, min_tokens=least)
    assert pkv.pkv_device_errors() == flags
    assert got.tolist() == want


@pytest.mark.parametrize("blocks", [255, 256, 2047, 2048, 2049, 5000])
def test_long_common_prefixes(blocks):
    row = list(range(blocks + 3))
    other = list(row)
    other[blocks - 1] = 1 << 20
    tables = [row, row, other, other, row]
    n = [(blocks + 2) * 16 + 3] * 5
    cu = list(range(6))
    want, _ = share_ref.shared_prefixes(cu, n, tables, 16, 1)
    wide = torch.full((5, blocks + 40), -5, dtype=torch.int32, device=DEV)
    wide[:, :blocks + 3] = i32(tables)
    assert pkv.pkv_shared_prefixes(i32(cu), i32(n), wide[:, :blocks + 3], 16, min_tokens=1).tolist() == want
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("wide", [0, 1000, 1100, 5000, 40000])
@pytest.mark.parametrize("B", [7, 8, 9, 17, 65, 200, 256, 257])
def test_groups_of_wide_tables(B, wide):
    """Tables much wider than what is used."""
    cu, n, tables = batch(B, B, 4, 6)
    want, flags = share_ref.shared_prefixes(cu, n, tables, 4, 4)
    t = torch.full((B, len(tables[0]) + wide), -9, dtype=torch.int32, device=DEV)
    t[:, :len(tables[0])] = i32(tables)
    assert pkv.pkv_shared_prefixes(i32(cu), i32(n), t, 4, 4).tolist() == want
    assert pkv.pkv_device_errors() == flags


@pytest.mark.parametrize("B", [2, 60, 256])
def test_first_differences_anywhere(B):
    """Tables that part at every place of a few trips."""
    r = random.Random(B)
    width = 1024 if B == 256 else 4000
    row = [r.randrange(1 << 20) for _ in range(width)]
    tables = []
    for s in range(B):
        row = list(row)
        at = r.choice([0, 1, 31, 32, 255, 256, 1023, 1024, 3000, width - 1, r.randrange(width)]) % width
        row[at] = (1 << 20) + s
        tables.append(row)
    n = [r.choice([width, width - 1, width // 2]) * 2 for _ in range(B)]
    cu = [0] * (B + 1)
    want, _ = share_ref.shared_prefixes(cu, n, tables, 2, 1)
    assert pkv.pkv_shared_prefixes(i32(cu), i32(n), i32(tables), 2, 1).tolist() == want
    assert pkv.pkv_device_errors() == 0


def test_bad_lengths_share_nothing():
    tables = [[1, 2, 3]] * 6
    for n, cu in (([8, 8, 13, 8, 8, 8], [0, 1, 2, 3, 4, 5, 6]), ([8, 8, -1, 8, 8, 8], [0, 1, 2, 3, 4, 5, 6]),
                  ([8, 8, 8, 8, 8, 8], [0, 1, 2, 12, 13, 14, 15]), ([8, 8, 8, 8, 8, 8], [0, 1, 3, 2, 4, 5, 6])):
        want, flags = share_ref.shared_prefixes(cu, n, tables, 4, 1)
        assert flags == 4
        assert pkv.pkv_shared_prefixes(i32(cu), i32(n), i32(tables), 4, 1).tolist() == want
        assert pkv.pkv_device_errors() == 4
    none = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    assert pkv.pkv_shared_prefixes(i32([0]), none[:, 0].contiguous(), torch.empty((0, 4), dtype=torch.int32, device=DEV), 4, 1).shape == (0, 3)


@pytest.mark.parametrize("B", [8191, 8192])
def test_groups_of_many_requests(B):
    cu, n, tables = batch(B, B, 4, 3)
    want, flags = share_ref.shared_prefixes(cu, n, tables, 4, 4)
    assert pkv.pkv_shared_prefixes(i32(cu), i32(n), i32(tables), 4, 4).tolist() == want
    assert pkv.pkv_device_errors() == flags
