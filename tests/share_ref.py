"""Plain references of the calls for requests that grow, shrink and share
prompts, written from their definitions, a request at a time, and a batch of
requests in groups."""
from tests.spec_ref import Batch


def step_tables(old, new, shared, bs, tables, free, count, T, width=None):
    """(tables, free, count, cu, slots, positions, error bits) after the step; tables and free are lists that are not
    changed."""
    B, F = len(old), len(free)
    width = len(tables[0]) if B else 0
    cap, flags = width * bs, 0
    up = lambda n: -(-n // bs)  # noqa: E731
    was_tables, was_free = [list(r) for r in tables], list(free)
    tables, free = [list(r) for r in tables], list(free)
    fine = []
    for a, b, sh in zip(old, new, shared):
        ok = 0 <= a <= cap and 0 <= b <= cap and 0 <= sh <= width and not (b > a and sh * bs > a)
        flags |= 0 if ok else 4
        fine.append(ok)
    rows = [max(0, b - a) if ok else 0 for a, b, ok in zip(old, new, fine)]
    refused = (was_tables, was_free, count, [0] * (B + 1), [-1] * T, [0] * T)
    if count < 0 or count > F or sum(rows) > T:
        return (*refused, flags | 4)
    stack = free[:count]
    for s in range(B):
        if fine[s]:
            stack += [tables[s][j] for j in range(max(up(new[s]), shared[s]), up(old[s]))]
    taken = sum(max(0, up(new[s]) - up(old[s])) for s in range(B) if fine[s])
    if taken > len(stack):
        return (*refused, flags | 32)
    if len(stack) - taken > F:
        return (*refused, flags | 4)
    for s in range(B):
        if fine[s]:
            for j in range(up(old[s]), up(new[s])):
                tables[s][j] = stack.pop()
    free[:len(stack)] = stack
    cu, slots, positions = [0], [], []
    for s in range(B):
        cu.append(cu[-1] + rows[s])
        for p in range(old[s], old[s] + rows[s]):
            block = tables[s][p // bs]
            if block < 0:
                flags |= 2
            slots.append(block * bs + p % bs if block >= 0 else -1)
            positions.append(p)
    pad = T - len(slots)
    return tables, free, len(stack), cu, slots + [-1] * pad, positions + [0] * pad, flags


def shared_prefixes(cu, n, tables, bs, least):
    """([first, end, prefix] of each request, error bits)."""
    B, flags, full = len(n), 0, []
    for s in range(B):
        q = cu[s + 1] - cu[s]
        ok = cu[s] >= 0 and 0 <= q <= n[s] and n[s] <= len(tables[s]) * bs
        flags |= 0 if ok else 4
        full.append((n[s] - q) // bs if ok else 0)
    common = [0] * (B + 1)
    for s in range(1, B):
        while common[s] < min(full[s], full[s - 1]) and tables[s][common[s]] == tables[s - 1][common[s]] >= 0:
            common[s] += 1
    link = [s > 0 and common[s] > 0 and common[s] * bs >= least and 2 * common[s] >= max(common[s - 1], common[s + 1]) for s in range(B)]
    out, s = [], 0
    while s < B:
        e = s + 1
        while e < B and link[e]:
            e += 1
        out += [[s, e, min(common[s + 1:e], default=0) * bs]] * (e - s)
        s = e
    return out, flags


class SharedBatch(Batch):
    """Requests in groups [(size, prefix tokens)] over a shuffled paged cache: own context tokens and new tokens of each.
    The requests of a group list the first one's blocks for their prefix."""

    def __init__(self, groups, own, q_lens, Hq, Hkv, D, bs, kv, seed, **kw):
        prefix = [p for size, p in groups for _ in range(size)]
        chain = [i - 1 for q in q_lens for i in range(q)]  # a chain of tokens sees what comes before: causal
        super().__init__([p + o for p, o in zip(prefix, own)], q_lens, Hq, Hkv, D, bs, kv, seed, parents=chain, **kw)
        at, self.groups = 0, []
        for size, p in groups:
            assert p % bs == 0
            self.groups += [[at, at + size, p]] * size
            for s in range(at, at + size):
                self.tables[s][:p // bs] = self.tables[at][:p // bs]
            at += size
        assert at == self.B
        self.max_group = max([int(self.cu[e] - self.cu[f]) for f, e, _ in self.groups] + [1])
