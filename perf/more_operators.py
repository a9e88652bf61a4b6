"""The operators of serving steps whose requests share prompts, as measured
cases: block tables and slots worked out on the GPU from the requests' lengths,
the shared prefixes that the tables hold, and attention that reads a shared
prefix once for all of its requests.

A case names sizes only; its lengths follow from "lens" (a seed that belongs to
the case) and its values from the seed given to prepare().
"""
import math
import random

import torch

own = False

CACHE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
CODE_SCALE = 1.0 / 96.0  # e4m3 caches: value = code * scale, so N(0, 1) rows use codes up to about 448


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the decode workload's batch: every request one token longer
        dict(name="tables decode B64", op="tables", B=64, bs=16, old_hi=4096, prompts=0.0, prompt_hi=1, ends=0.0, cuts=0.0, grow=1,
             shared=0, lens=41),
        # a speculative step with odd blocks: drafts of up to 8 tokens appended, rejected ones given back, some requests done
        dict(name="tables drafts B37 bs12", op="tables", B=37, bs=12, old_hi=3001, prompts=0.1, prompt_hi=700, ends=0.1, cuts=0.4, grow=8,
             shared=60, lens=42),
        # a busy server: prompts admitted behind a shared system prompt, requests done, the rest decode
        dict(name="tables prompts B256", op="tables", B=256, bs=16, old_hi=16384, prompts=0.1, prompt_hi=2048, ends=0.1, cuts=0.1, grow=4,
             shared=1024, lens=43),
        # one system prompt in front of a decode batch
        dict(name="prefixes B64 p2048", op="prefixes", B=64, bs=16, g_lo=64, g_hi=64, p_lo=2048, p_hi=2048, alone=0.0, s_lo=64, s_hi=2048,
             q_lo=1, q_hi=1, least=256, lens=51),
        # many documents, several questions about each, some long
        dict(name="prefixes B256 uneven", op="prefixes", B=256, bs=16, g_lo=1, g_hi=24, p_lo=16, p_hi=65536, alone=0.2, s_lo=0, s_hi=2048,
             q_lo=1, q_hi=4, least=256, lens=52),
        # a few samples of one short prompt: latency
        dict(name="shared B4 p1024", op="shared", B=4, g_lo=4, g_hi=4, p_lo=1024, p_hi=1024, alone=0.0, s_lo=16, s_hi=128, q_lo=1, q_hi=1,
             Hq=32, Hkv=8, D=128, cache="bf16", bs=16, lens=61),
        # the decode workload's batch and heads behind one system prompt
        dict(name="shared B64 p2048", op="shared", B=64, g_lo=64, g_hi=64, p_lo=2048, p_hi=2048, alone=0.0, s_lo=512, s_hi=2048, q_lo=1, q_hi=1,
             Hq=32, Hkv=8, D=128, cache="bf16", bs=16, lens=62),
        # questions about documents: groups of uneven size, some requests alone
        dict(name="shared B64 documents", op="shared", B=64, g_lo=2, g_hi=12, p_lo=1024, p_hi=8192, alone=0.2, s_lo=64, s_hi=1024, q_lo=1,
             q_hi=1, Hq=32, Hkv=8, D=128, cache="bf16", bs=16, lens=63),
        # the long-context batch on fp8 caches, about one text
        dict(name="shared B16 e4m3 long", op="shared", B=16, g_lo=16, g_hi=16, p_lo=65536, p_hi=65536, alone=0.0, s_lo=512, s_hi=4096, q_lo=1,
             q_hi=1, Hq=32, Hkv=8, D=128, cache="e4m3", bs=16, lens=64),
        # many samples of many prompts on fp8 caches
        dict(name="shared B256 e4m3", op="shared", B=256, g_lo=16, g_hi=16, p_lo=512, p_hi=2048, alone=0.0, s_lo=64, s_hi=1024, q_lo=1, q_hi=1,
             Hq=32, Hkv=8, D=128, cache="e4m3", bs=16, lens=65),
        # odd everything: five heads for each KV head, D 64, blocks of 12, one to seven rows a request
        dict(name="shared odd D64 G5", op="shared", B=23, g_lo=1, g_hi=9, p_lo=12, p_hi=3001, alone=0.3, s_lo=0, s_hi=501, q_lo=1, q_hi=7,
             Hq=15, Hkv=3, D=64, cache="bf16", bs=12, lens=66),
        # chunks of prompts behind a shared system prompt
        dict(name="shared chunks B16 q64", op="shared", B=16, g_lo=16, g_hi=16, p_lo=4096, p_hi=4096, alone=0.0, s_lo=0, s_hi=256, q_lo=64,
             q_hi=64, Hq=32, Hkv=8, D=128, cache="bf16", bs=16, lens=67),
    ]


def _log(rng, a, b):
    """A whole number spread over a .. b by its logarithm."""
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["tables", "tables", "prefixes", "shared", "shared", "shared", "shared"])
    lens = rng.randrange(1 << 20)
    bs = rng.choice([1, 4, 8, 12, 16, 32, 64])
    if op == "tables":
        return dict(op=op, B=_log(rng, 1, 256), bs=bs, old_hi=_log(rng, 16, 16384), prompts=rng.choice([0.0, 0.1, 0.3]),
                    prompt_hi=_log(rng, 1, 2048), ends=rng.choice([0.0, 0.1, 0.5]), cuts=rng.choice([0.0, 0.2]), grow=rng.randint(1, 16),
                    shared=rng.choice([0, bs * rng.randint(1, 16)]), lens=lens)
    if op == "prefixes":
        B, p = _log(rng, 8, 256), _log(rng, 256, 65536)
        return dict(op=op, B=B, bs=max(bs, 4), g_lo=1, g_hi=_log(rng, 2, B), p_lo=rng.choice([p, p // 4]), p_hi=p, alone=rng.choice([0.0, 0.2]),
                    s_lo=0, s_hi=_log(rng, 16, 2048), q_lo=1, q_hi=_log(rng, 1, 16), least=_log(rng, 16, 256), lens=lens)
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    q1 = rng.choice([1, 1, 1, _log(rng, 2, 64)])
    p1 = _log(rng, 64, 65536)
    s1 = _log(rng, 16, 4096)
    # no more keys in all, counted for each request, and no more scores, than the largest listed cases have
    B = max(1, min(_log(rng, 1, 256), 800000 // (p1 + s1), 400000000 // ((p1 + s1) * q1 * Hkv * G)))
    return dict(op=op, B=B, g_lo=1, g_hi=_log(rng, 1, B), p_lo=rng.choice([p1, p1 // 4]), p_hi=p1, alone=rng.choice([0.0, 0.0, 0.3]),
                s_lo=rng.choice([0, s1 // 2]), s_hi=s1, q_lo=rng.choice([1, q1]), q_hi=q1, Hq=Hkv * G, Hkv=Hkv, D=D,
                cache=rng.choice(["bf16", "e4m3"]), bs=bs, lens=lens)


def _changes(case):
    """(length before, length after, shared blocks) of each request: plain lists that follow from the case alone."""
    r = random.Random(case["lens"])
    bs, old, new, shared = case["bs"], [], [], []
    for _ in range(case["B"]):
        u = r.random()
        sh = case["shared"] // bs if r.random() < 0.5 else 0
        a = sh * bs + r.randint(0, case["old_hi"])
        if u < case["prompts"]:  # admitted: its cached prefix is there, the prompt's tokens come
            a = sh * bs
            b = a + r.randint(1, case["prompt_hi"])
        elif u < case["prompts"] + case["ends"]:
            b = 0
        elif u < case["prompts"] + case["ends"] + case["cuts"]:  # drafted tokens that were rejected
            b = max(sh * bs, a - r.randint(0, 16))
        else:
            b = a + r.randint(1, case["grow"])
        old.append(a)
        new.append(b)
        shared.append(sh)
    return old, new, shared


def _batch(case, seed=0):
    """(size, prefix tokens) of each group of requests and (own context tokens, new tokens) of each request.  Where
    the lengths are the inputs (prefixes) they follow from the seed too."""
    r = random.Random(case["lens"] + (seed << 20 if case["op"] == "prefixes" else 0))
    bs, groups, left = case["bs"], [], case["B"]
    while left:
        n = min(left, r.randint(case["g_lo"], case["g_hi"]))
        n = 1 if r.random() < case["alone"] else n
        p = r.randint(case["p_lo"], case["p_hi"]) // bs * bs
        groups.append((n, 0 if n == 1 and case["op"] == "shared" else p))
        left -= n
    return groups, [(r.randint(case["s_lo"], case["s_hi"]), r.randint(case["q_lo"], case["q_hi"])) for _ in range(case["B"])]


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(gen, blocks, bs, Hkv, D, cache):
    """A cache of N(0, 1) rows."""
    out = torch.empty((blocks, bs, Hkv, D), dtype=CACHE[cache], device="cuda")
    flat = out.view(blocks, -1)
    step = max(1, (1 << 28) // max(1, flat.shape[1]))
    for b in range(0, blocks, step):
        x = torch.randn((min(step, blocks - b), flat.shape[1]), generator=gen, device="cuda")
        flat[b:b + step] = (x if cache == "bf16" else (x / CODE_SCALE).clamp(-448, 448)).to(CACHE[cache])
    return out


def _tables(perm, used, first, width):
    """Tables of `used` blocks each, taken from perm at `first`; -1 behind them."""
    col = torch.arange(width, device="cuda")
    n, at = torch.tensor(used, device="cuda"), torch.tensor(first, device="cuda")
    got = perm[(at[:, None] + col[None, :]).clamp(max=perm.shape[0] - 1)]
    return torch.where(col[None, :] < n[:, None], got, torch.tensor(-1, dtype=torch.int32, device="cuda"))


def _summed(n):
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    return at


def _blocks(n, bs):
    return -(-n // bs)


def _prepare_tables(case, gen):
    old, new, shared = _changes(case)
    bs = case["bs"]
    used = [_blocks(n, bs) for n in old]
    at = _summed(used)
    taken = sum(max(0, _blocks(b, bs) - _blocks(a, bs)) for a, b in zip(old, new))
    pool = at[-1] + taken + 64
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    width = max(_blocks(max(a, b), bs) for a, b in zip(old, new)) + 3
    T = sum(max(0, b - a) for a, b in zip(old, new))
    free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    free[:pool - at[-1]] = perm[at[-1]:]
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "T": T, "old": _i32(old), "new": _i32(new), "shared": _i32(shared), "bt": _tables(perm, used, at[:-1], width),
            "free": free, "count": _i32([pool - at[-1]]), "new_count": i32(1), "cu": i32(case["B"] + 1), "slots": i32(T), "positions": i32(T)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, gen)
    groups, rows = _batch(case, seed)
    bs, st = case["bs"], {"case": case}
    prefix = [p for n, p in groups for _ in range(n)]
    n = [p + s + q for p, (s, q) in zip(prefix, rows)]
    # a group's prefix is stored once, in front of the blocks of its requests
    first, own_first, at = [], [], 0
    for (size, p), lo in zip(groups, _summed([g for g, _ in groups])):
        mine = at
        at += p // bs
        for s in range(lo, lo + size):
            first.append(mine)
            own_first.append(at)
            at += _blocks(n[s], bs) - p // bs
    perm = torch.randperm(at + 7, generator=gen, device="cuda").to(torch.int32)
    width = max(_blocks(m, bs) for m in n) if case["op"] == "shared" else _blocks(case["p_hi"] + case["s_hi"] + case["q_hi"], bs)
    used = [_blocks(m, bs) for m in n]
    head = torch.tensor([p // bs for p in prefix], device="cuda")[:, None]
    shift = (torch.tensor(own_first, device="cuda")[:, None] - head)
    col = torch.arange(width, device="cuda")[None, :]
    idx = torch.where(col < head, torch.tensor(first, device="cuda")[:, None] + col, shift + col).clamp(max=at + 6)
    st["bt"] = torch.where(col < torch.tensor(used, device="cuda")[:, None], perm[idx], torch.tensor(-1, dtype=torch.int32, device="cuda"))
    cu = _summed([q for _, q in rows])
    st["cu"], st["n"], st["T"] = _i32(cu), _i32(n), cu[-1]
    st["max_q"], st["max_n"] = max(q for _, q in rows), max(n)
    if case["op"] == "prefixes":
        # one request in eight leaves its group's prefix early: from some block on its blocks are its own
        u = torch.rand((2, case["B"], 1), generator=gen, device="cuda", dtype=torch.float64)
        leave = torch.where(u[0] < 0.125, (u[1] * (head + 1)).long(), width)
        st["bt"] = torch.where((col >= leave) & (st["bt"] >= 0), st["bt"] + (at + 7) * (1 + torch.arange(case["B"], device="cuda")[:, None]),
                               st["bt"]).to(torch.int32)
        st["groups"] = torch.empty((case["B"], 3), dtype=torch.int32, device="cuda")
        return st
    lo = _summed([g for g, _ in groups])
    st["max_group"] = max(cu[b] - cu[a] for a, b in zip(lo, lo[1:]))
    st["groups"] = _i32([[a, a + g, p] for (g, p), a in zip(groups, lo) for _ in range(g)])
    st["kc"] = _cache(gen, at + 7, bs, case["Hkv"], case["D"], case["cache"])
    st["vc"] = _cache(gen, at + 7, bs, case["Hkv"], case["D"], case["cache"])
    st["q"] = (1.5 * torch.randn((cu[-1], case["Hq"], case["D"]), generator=gen, device="cuda")).to(torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    return st


# ---------------------------------------------------------------- plain forms
def _rows(cu, T):
    """(sequence, index in it) of each packed row."""
    cu = cu.long()
    t = torch.arange(T, device=cu.device)
    s = torch.searchsorted(cu, t, right=True) - 1
    return s, t - cu[s]


def _up(n, bs):
    return (n + bs - 1) // bs


def _plain_tables(st):
    bs, T = st["case"]["bs"], st["T"]
    old, new, shared, bt = st["old"].long(), st["new"].long(), st["shared"].long(), st["bt"].long()
    q = (new - old).clamp(min=0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(q, 0)])
    b0, b1 = _up(old, bs), _up(new, bs)
    take = (b1 - b0).clamp(min=0)
    kept = torch.maximum(b1, shared)
    col = torch.arange(bt.shape[1], device="cuda")[None, :]
    back = bt[(col >= kept[:, None]) & (col < b0[:, None])]  # blocks given back, by request and place
    count = st["count"].long()
    at = torch.arange(st["free"].shape[0], device="cuda")
    pad = torch.cat([back, torch.full((1,), -1, dtype=torch.int64, device="cuda")])
    stack = torch.where(at < count, st["free"].long(), pad[(at - count).clamp(0, back.shape[0])])
    order = (torch.cumsum(take, 0) - take - b0)[:, None] + col  # which of the taken blocks a column gets
    top = count + back.shape[0]
    got = stack[(top - 1 - order).clamp(0, at.shape[0] - 1)]
    bt = torch.where((col >= b0[:, None]) & (col < b1[:, None]), got, bt)
    left = top - take.sum()
    s, i = _rows(cu, T)
    pos = old[s] + i
    st["free"].copy_(torch.where(at < left, stack, st["free"].long()))
    st["bt"].copy_(bt)
    return {"block_tables": st["bt"], "free_blocks": st["free"], "free_count": left.to(torch.int32), "cu_seqlens_q": cu.to(torch.int32),
            "slots": (bt[s, pos // bs] * bs + pos % bs).to(torch.int32), "positions": pos.to(torch.int32)}


def _plain_prefixes(st):
    c = st["case"]
    B, bs = c["B"], c["bs"]
    cu, n, bt = st["cu"].long(), st["n"].long(), st["bt"]
    full = (n - (cu[1:] - cu[:-1])) // bs  # whole blocks of context
    col = torch.arange(bt.shape[1], device="cuda")[None, :]
    same = (bt[1:] == bt[:-1]) & (bt[1:] >= 0) & (col < torch.minimum(full[1:], full[:-1])[:, None])
    common = torch.zeros(B + 1, dtype=torch.int64, device="cuda")  # leading blocks that a request shares with the one before
    common[1:B] = torch.where(same, col.shape[1], col).amin(1)
    mine, prev, after = common[:B], common[:-1].roll(1), common[1:]
    prev = torch.where(torch.arange(B, device="cuda") == 0, 0, prev)
    link = (mine * bs >= c["least"]) & (mine > 0) & (2 * mine >= torch.maximum(prev, after))
    g = torch.cumsum((~link).long(), 0) - 1
    at = torch.arange(B, device="cuda")
    first = torch.full((B,), B, dtype=torch.int64, device="cuda").scatter_reduce(0, g, at, "amin")
    last = torch.zeros(B, dtype=torch.int64, device="cuda").scatter_reduce(0, g, at, "amax")
    least = torch.full((B,), 1 << 40, dtype=torch.int64, device="cuda").scatter_reduce(0, g, torch.where(link, mine, 1 << 40), "amin")
    prefix = torch.where(least < 1 << 40, least * bs, 0)
    return torch.stack([first[g], last[g] + 1, prefix[g]], 1).to(torch.int32)


def _gathered(cache, slot, scale):
    """Rows of a cache in 32 bits, by slot."""
    _, _, Hkv, D = cache.shape
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8).view(-1, Hkv, D)[slot].view(torch.float8_e4m3fn).float() * scale
    return cache.view(-1, Hkv, D)[slot].float()


def _plain_shared(st):
    """Causal attention of every request over its own table."""
    c, T, max_q, max_n = st["case"], st["T"], st["max_q"], st["max_n"]
    B, Hq, Hkv, D, bs = c["B"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    G = Hq // Hkv
    cu, n, bt = st["cu"].long(), st["n"].long(), st["bt"].long()
    j = torch.arange(max_n, device="cuda")
    slot = (bt[:, j // bs].clamp(min=0) * bs + (j % bs)[None, :])
    k = _gathered(st["kc"], slot, CODE_SCALE).permute(0, 2, 3, 1)  # [B, Hkv, D, N]
    i = torch.arange(max_q, device="cuda")
    q_len = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)  # [B, max_q]
    q = st["q"][row].float().view(B, max_q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, max_q * G, D)
    x = torch.matmul(q, k).view(B, Hkv, max_q, G, max_n) * D ** -0.5
    del k
    seen = j[None, None, :] <= ((n - q_len)[:, None] + i[None, :])[:, :, None]  # [B, max_q, N]
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _gathered(st["vc"], slot, CODE_SCALE).permute(0, 2, 1, 3)  # [B, Hkv, N, D]
    o = torch.matmul(x.view(B, Hkv, max_q * G, max_n), v).view(B, Hkv, max_q, G, D) / total
    s, at_q = _rows(cu, T)
    return o.permute(0, 2, 1, 3, 4).reshape(B, max_q, Hq, D)[s, at_q].to(st["q"].dtype)


# ---------------------------------------------------------------- one pass
def _kept(st, name, make):
    """What a program makes once and keeps: a workspace."""
    if name not in st:
        st[name] = make()
    return st[name]


def _own(st):
    import paged_kv_cache_mapping_gb300 as pkv
    c = st["case"]
    if c["op"] == "tables":
        pkv.pkv_step_tables(st["old"], st["new"], st["bt"], c["bs"], st["free"], st["count"], st["cu"], st["slots"],
                            shared_blocks=st["shared"], positions=st["positions"], new_free_count=st["new_count"])
        return {"block_tables": st["bt"], "free_blocks": st["free"], "free_count": st["new_count"].view(()), "cu_seqlens_q": st["cu"],
                "slots": st["slots"], "positions": st["positions"]}
    if c["op"] == "prefixes":
        return pkv.pkv_shared_prefixes(st["cu"], st["n"], st["bt"], c["bs"], min_tokens=c["least"], groups=st["groups"])
    scale = CODE_SCALE if c["cache"] == "e4m3" else 1.0
    ws = _kept(st, "ws", lambda: torch.empty(
        pkv.pkv_shared_attention_workspace_size(st["q"], st["bt"], st["kc"], st["max_q"], st["max_group"]), dtype=torch.uint8, device="cuda"))
    return pkv.pkv_shared_attention(st["q"], st["cu"], st["n"], st["bt"], st["groups"], st["kc"], st["vc"], c["D"] ** -0.5, st["out"],
                                    k_scale=scale, v_scale=scale, max_q_len=st["max_q"], max_group_len=st["max_group"], workspace=ws)


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "tables":
        out = _plain_tables(st)
        return {**out, "free_count": out["free_count"].view(())}
    if op == "prefixes":
        return _plain_prefixes(st)
    return _plain_shared(st)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    bs = case["bs"]
    if case["op"] == "tables":
        old, new, shared = _changes(case)
        T = sum(max(0, b - a) for a, b in zip(old, new))
        taken = sum(max(0, _blocks(b, bs) - _blocks(a, bs)) for a, b in zip(old, new))
        back = sum(max(0, _blocks(a, bs) - max(_blocks(b, bs), sh)) for a, b, sh in zip(old, new, shared))
        # lengths in, rows' slots and positions out; a block moves from the list to a table, or back
        return {"bytes": 16 * case["B"] + 8 * T + 8 * (taken + back) + 8, "flops": T}
    groups, rows = _batch(case)
    prefix = [p for n, p in groups for _ in range(n)]
    if case["op"] == "prefixes":
        return {"bytes": 20 * case["B"] + 4 * sum(p // bs for p in prefix), "flops": sum(p // bs for p in prefix)}
    es = 1 if case["cache"] == "e4m3" else 2
    Hkv, D, Hq = case["Hkv"], case["D"], case["Hq"]
    keys = sum(p for _, p in groups) + sum(s + q for s, q in rows)
    T = sum(q for _, q in rows)
    seen = sum(q * (p + s) + q * (q + 1) // 2 for p, (s, q) in zip(prefix, rows))
    return {"bytes": 2 * keys * Hkv * D * es + 4 * T * Hq * D + 4 * (keys // bs) + 24 * case["B"], "flops": 4 * D * Hq * seen}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    if case["op"] != "shared":
        return None  # whole numbers
    st = prepare(case, seed)
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    s = CODE_SCALE if case["cache"] == "e4m3" else 1.0
    cu, n = st["cu"].tolist(), st["n"].tolist()
    out = torch.zeros((cu[-1], Hq, D), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        m = cu[b + 1] - cu[b]
        blocks = st["bt"][b, :_blocks(n[b], bs)].long()
        k, v = (x[blocks].reshape(-1, Hkv, D)[:n[b]].double() * s for x in (st["kc"], st["vc"]))
        hidden = torch.ones((m, n[b]), dtype=torch.bool, device="cuda").triu(n[b] - m + 1)
        for h in range(Hkv):
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            e = torch.einsum("igd,jd->igj", st["q"][cu[b]:cu[b + 1], mine].double(), k[:, h]) * D ** -0.5
            out[cu[b]:cu[b + 1], mine] = torch.einsum("igj,jd->igd", torch.softmax(e.masked_fill(hidden[:, None, :], -math.inf), -1), v[:, h])
    return out
