"""The operators of a speculative decoding step over the paged KV cache, as
measured cases: rotary positions with the cache append, the mask of a tree of
drafted tokens, attention of the tree over the cache, and the compaction of
the accepted path's rows.

A case names sizes only; its sequence lengths follow from "lens" (a seed that
belongs to the case) and its values from the seed given to prepare().
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
        # one decode step's rows, Qwen3-4B heads: latency
        dict(name="rope decode B64", op="rope", T=64, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             scaling="none", max_pos=4096, cache="bf16", bs=16, blocks=1024),
        # the rows of drafted trees at far positions: part of the head, pairs side by side, long-context ramp, fp8 cache
        dict(name="rope drafts e4m3 far", op="rope", T=777, Hq=20, Hkv=5, D=64, rot=48, interleaved=True,
             scaling="by_parts", max_pos=1000000, cache="e4m3", bs=16, blocks=1024),
        # a prompt's chunk of rows
        dict(name="rope prompt T8192", op="rope", T=8192, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             scaling="smooth", max_pos=131072, cache="bf16", bs=16, blocks=1024),
        # small trees of one batch; large and uneven ones
        dict(name="mask B64 q16", op="mask", B=64, q_lo=16, q_hi=16, ctx_lo=0, ctx_hi=4096, lens=11),
        dict(name="mask B256 q1-100", op="mask", B=256, q_lo=1, q_hi=100, ctx_lo=0, ctx_hi=4096, lens=12),
        # one user, a small tree on a short context: latency
        dict(name="tree B1 q8 ctx2048", op="tree", B=1, q_lo=8, q_hi=8, ctx_lo=2048, ctx_hi=2048, Hq=32, Hkv=8, D=128,
             cache="bf16", bs=16, holes=False, lens=21),
        # the decode workload's batch with eight drafted tokens each
        dict(name="tree B64 q8 ctx512-4096", op="tree", B=64, q_lo=8, q_hi=8, ctx_lo=512, ctx_hi=4096, Hq=32, Hkv=8, D=128,
             cache="bf16", bs=16, holes=False, lens=22),
        # wide trees: 256 query rows for each KV head
        dict(name="tree B16 q64 ctx1024-8192", op="tree", B=16, q_lo=64, q_hi=64, ctx_lo=1024, ctx_hi=8192, Hq=32, Hkv=8, D=128,
             cache="bf16", bs=16, holes=False, lens=23),
        # the long-context batch on fp8 caches
        dict(name="tree B8 q16 e4m3 long", op="tree", B=8, q_lo=16, q_hi=16, ctx_lo=32768, ctx_hi=131072, Hq=32, Hkv=8, D=128,
             cache="e4m3", bs=16, holes=False, lens=24),
        # odd everything: uneven trees, five heads for each KV head, D 64, blocks of 12, masks with empty rows
        dict(name="tree odd D64 G5", op="tree", B=23, q_lo=1, q_hi=37, ctx_lo=0, ctx_hi=3001, Hq=15, Hkv=3, D=64,
             cache="bf16", bs=12, holes=True, lens=25),
        # accepted paths after a verification step
        dict(name="commit B64 path8", op="commit", B=64, q_lo=16, q_hi=16, path=8, ctx_lo=0, ctx_hi=200, Hkv=8, D=128,
             cache="bf16", bs=16, lens=31),
        dict(name="commit B256 path5 e4m3", op="commit", B=256, q_lo=9, q_hi=40, path=5, ctx_lo=0, ctx_hi=100, Hkv=5, D=64,
             cache="e4m3", bs=12, lens=32),
    ]


def _log(rng, a, b):
    """A whole number spread over a .. b by its logarithm."""
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["rope", "mask", "tree", "tree", "tree", "commit"])
    cache = rng.choice(["bf16", "e4m3"])
    lens = rng.randrange(1 << 20)
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    bs = rng.choice([1, 4, 8, 12, 16, 32, 64])
    if op == "rope":
        T = _log(rng, 1, 8192)
        interleaved = rng.random() < 0.5
        return dict(op=op, T=T, Hq=Hkv * min(G, 4), Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D // 2 - 8, 2 * rng.randint(1, D // 2)]),
                    interleaved=interleaved, scaling=rng.choice(["none", "linear", "ntk", "by_parts", "smooth"]),
                    max_pos=_log(rng, 4096, 1000000), cache=cache, bs=bs, blocks=-(-T // bs) + rng.randint(1, 64))
    if op == "mask":
        hi = _log(rng, 1, 128)
        return dict(op=op, B=_log(rng, 1, 256), q_lo=rng.randint(1, hi), q_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 16, 131072), lens=lens)
    if op == "commit":
        path = rng.randint(1, 12)
        return dict(op=op, B=_log(rng, 1, 256), q_lo=path, q_hi=path + rng.randint(0, 60), path=path, ctx_lo=0, ctx_hi=_log(rng, 16, 256),
                    Hkv=Hkv, D=D, cache=cache, bs=bs, lens=lens)
    q1 = _log(rng, 1, 100)
    q0 = rng.choice([q1, rng.randint(1, q1)])
    ctx1 = _log(rng, 64, 131072)
    ctx0 = rng.choice([0, ctx1 // 8, ctx1 // 2])
    B = _log(rng, 1, 64)
    # no more keys in all, and no more scores, than the largest listed cases have
    B = max(1, min(B, 300000 // ctx1, 500000000 // (ctx1 * q1 * Hkv * G)))
    return dict(op="tree", B=B, q_lo=q0, q_hi=q1, ctx_lo=ctx0, ctx_hi=ctx1, Hq=Hkv * G, Hkv=Hkv, D=D, cache=cache, bs=bs,
                holes=rng.random() < 0.3, lens=lens)


def _lengths(case):
    """(context tokens, drafted tokens) of each sequence: plain lists that follow from the case alone."""
    r = random.Random(case["lens"])
    return ([r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])],
            [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])])


# ---------------------------------------------------------------- inputs
def _rope_settings(case):
    s = dict(rot_dim=case["rot"], base=1000000.0 if case["max_pos"] > 32768 else 10000.0, interleaved=case["interleaved"],
             scaling=case["scaling"])
    if case["scaling"] != "none":
        s["factor"] = 8.0
    if case["scaling"] in ("by_parts", "smooth"):
        s["original_max_position"] = max(2048, case["max_pos"] // 8)
    return s


def _cache(gen, blocks, bs, Hkv, D, cache):
    """A cache of N(0, 1) rows."""
    out = torch.empty((blocks, bs, Hkv, D), dtype=CACHE[cache], device="cuda")
    flat = out.view(blocks, -1)
    step = max(1, (1 << 28) // max(1, flat.shape[1]))
    for b in range(0, blocks, step):
        x = torch.randn((min(step, blocks - b), flat.shape[1]), generator=gen, device="cuda")
        flat[b:b + step] = (x if cache == "bf16" else (x / CODE_SCALE).clamp(-448, 448)).to(CACHE[cache])
    return out


def _tables(gen, tokens, bs):
    """Block tables over a shuffled pool, and the pool's size."""
    need = [-(-n // bs) for n in tokens]
    pool = sum(need) + 7
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    width = max(need + [1])
    col = torch.arange(width, device="cuda")
    n = torch.tensor(need, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = first[:, None] + col[None, :]
    return torch.where(col[None, :] < n[:, None], perm[at.clamp(max=pool - 1)], torch.tensor(-1, dtype=torch.int32, device="cuda")), pool


def _cu(q):
    at = [0]
    for n in q:
        at.append(at[-1] + n)
    return at


def _trees(gen, cu):
    """Parents of random trees: every node but the first hangs off an earlier one."""
    T = cu[-1]
    cu_t = torch.tensor(cu, device="cuda")
    t = torch.arange(T, device="cuda")
    i = t - cu_t[torch.searchsorted(cu_t, t, right=True) - 1]
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64).pow(0.5)
    return torch.where(i == 0, -1, torch.minimum((u * i).long(), i - 1)).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "rope":
        T, Hq, Hkv, D, bs = case["T"], case["Hq"], case["Hkv"], case["D"], case["bs"]
        n = case["blocks"] * bs
        st["q"] = torch.randn((T, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
        st["k"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
        st["v"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
        st["positions"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        st["slots"] = torch.randperm(n, generator=gen, device="cuda")[:T].to(torch.int32)
        st["kc"] = _cache(gen, case["blocks"], bs, Hkv, D, case["cache"])
        st["vc"] = _cache(gen, case["blocks"], bs, Hkv, D, case["cache"])
        st["q_out"] = torch.empty_like(st["q"])
        st["rope"] = _rope_settings(case)
        return st
    ctx, q = _lengths(case)
    cu = _cu(q)
    n = [a + b for a, b in zip(ctx, q)]
    st["T"], st["max_q"], st["max_n"] = cu[-1], max(q), max(n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["n"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    if case["op"] == "mask":
        st["parents"] = _trees(gen, cu)
        return st
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    st["bt"], pool = _tables(gen, n, bs)
    st["kc"] = _cache(gen, pool, bs, Hkv, D, case["cache"])
    st["vc"] = _cache(gen, pool, bs, Hkv, D, case["cache"])
    if case["op"] == "commit":
        # paths of 1 .. path nodes, ascending: the first entries of a sorted sample of the tree
        B, A = case["B"], case["path"]
        q_t = torch.tensor(q, device="cuda")
        u = torch.rand((B, max(q)), generator=gen, device="cuda")
        u = torch.where(torch.arange(max(q), device="cuda")[None, :] < q_t[:, None], u, 2.0)
        st["accepted"] = u.argsort(dim=1)[:, :A].sort(dim=1).values.to(torch.int32).contiguous()
        st["accepted_lens"] = torch.randint(1, A + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        st["new_n"] = torch.empty_like(st["n"])
        return st
    T = cu[-1]
    st["q"] = (1.5 * torch.randn((T, case["Hq"], D), generator=gen, device="cuda")).to(torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    words = -(-max(q) // 32)
    bits, _ = _plain_mask(_trees(gen, cu), st["cu"], st["n"], T, max(q))
    if case["holes"]:  # general masks: some bits dropped, some rows without any
        drop = torch.randint(0, 1 << 32, bits.shape, generator=gen, device="cuda").to(torch.int32)
        bits = bits & drop
    st["mask"] = bits[:, :words].contiguous()
    return st


# ---------------------------------------------------------------- plain forms
def _rows(cu, T):
    """(sequence, index in it) of each packed row."""
    cu = cu.long()
    t = torch.arange(T, device=cu.device)
    s = torch.searchsorted(cu, t, right=True) - 1
    return s, t - cu[s]


def _frequencies(rot, base, scaling, factor=1.0, original_max_position=0, dtype=torch.float64):
    """Angles per position of the rotated pairs, and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=dtype, device="cuda")
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    f = torch.pow(torch.tensor(base, dtype=dtype, device="cuda"), -2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":  # fast pairs keep their angles, slow ones are stretched, a ramp between 32 turns and 1
        at = lambda turns: rot * math.log(original_max_position / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    if scaling == "smooth":  # the same by the turns over the original length: 4 and more, 1 and fewer
        turns = original_max_position * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    return f, 1.0


def _rotate(x, cos, sin, rot, interleaved):
    x, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:]
        x = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([x, rest], -1)


def _store(cache, slots, rows):
    """Rows (32 bits) into their slots, in the cache's type."""
    _, _, Hkv, D = cache.shape
    if cache.dtype == torch.float8_e4m3fn:
        codes = (rows * (1.0 / CODE_SCALE)).clamp(-448, 448).to(torch.float8_e4m3fn)
        cache.view(torch.uint8).view(-1, Hkv, D)[slots] = codes.view(torch.uint8)
    else:
        cache.view(-1, Hkv, D)[slots] = rows.to(cache.dtype)


def _plain_rope(st):
    r = st["rope"]
    f, m = _frequencies(r["rot_dim"], r["base"], r["scaling"], r.get("factor", 1.0), r.get("original_max_position", 0))
    angle = st["positions"].double()[:, None] * f[None, :]  # 64 bits: a far position has millions of turns
    cos, sin = (m * angle.cos()).float()[:, None, :], (m * angle.sin()).float()[:, None, :]
    q = _rotate(st["q"].float(), cos, sin, r["rot_dim"], r["interleaved"]).to(st["q"].dtype)
    slots = st["slots"].long()
    _store(st["kc"], slots, _rotate(st["k"].float(), cos, sin, r["rot_dim"], r["interleaved"]))
    _store(st["vc"], slots, st["v"].float())
    return {"q": q, "k_cache": st["kc"], "v_cache": st["vc"]}


def _plain_mask(parents, cu, n, T, max_q):
    """(mask words, positions): node i sees its ancestors and itself."""
    B = n.shape[0]
    s, i = _rows(cu, T)
    child = torch.zeros((B, max_q, max_q), device="cuda")
    p = parents.long()
    child[s, i, p.clamp(min=0)] = (p >= 0).float()
    eye = torch.eye(max_q, device="cuda")
    sees = child + eye
    for _ in range(max(1, max_q - 1).bit_length()):  # paths of 1, 2, 4, .. steps
        sees = (torch.matmul(sees, sees) > 0).float()
    seen = sees[s, i]  # [T, max_q]
    depth = seen.sum(1).long() - 1
    words = -(-max_q // 32)
    bits = torch.zeros((T, words * 32), dtype=torch.int64, device="cuda")
    bits[:, :max_q] = seen.long()
    value = (bits.view(T, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    value = torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)
    ctx = (n.long() - (cu[1:] - cu[:-1]).long())[s]
    return value, (ctx + depth).to(torch.int32)


def _gathered(cache, slot, scale):
    """Rows of a cache in 32 bits, by slot."""
    _, _, Hkv, D = cache.shape
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8).view(-1, Hkv, D)[slot].view(torch.float8_e4m3fn).float() * scale
    return cache.view(-1, Hkv, D)[slot].float()


def _plain_tree(st):
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
    at = j[None, :] - (n - q_len)[:, None]  # drafted index of each key, negative in the context
    word = st["mask"].long()[row]  # [B, max_q, words]
    word = torch.gather(word, 2, (at.clamp(0, max_q - 1) // 32)[:, None, :].expand(B, max_q, max_n))
    bit = ((word >> (at.clamp(min=0) % 32)[:, None, :]) & 1) > 0
    seen = (at[:, None, :] < 0) | (bit & (at < q_len[:, None])[:, None, :])
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _gathered(st["vc"], slot, CODE_SCALE).permute(0, 2, 1, 3)  # [B, Hkv, N, D]
    o = torch.matmul(x.view(B, Hkv, max_q * G, max_n), v).view(B, Hkv, max_q, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(B, max_q, Hq, D)
    s, at_q = _rows(cu, T)
    return o[s, at_q].to(st["q"].dtype)


def _plain_commit(st):
    c = st["case"]
    Hkv, D, bs, A = c["Hkv"], c["D"], c["bs"], c["path"]
    cu, n = st["cu"].long(), st["n"].long()
    base = n - (cu[1:] - cu[:-1])
    i = torch.arange(A, device="cuda")[None, :]
    kept = i < st["accepted_lens"][:, None]
    src = base[:, None] + torch.where(kept, st["accepted"].long(), i)  # entries past the path stay where they are
    dst = base[:, None] + i
    bt = st["bt"].long()
    src = torch.gather(bt, 1, src // bs) * bs + src % bs
    dst = torch.gather(bt, 1, dst // bs) * bs + dst % bs
    k, v = (t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8).view(-1, Hkv, D) for t in (st["kc"], st["vc"]))
    k[dst] = k[src]
    v[dst] = v[src]
    return {"k_cache": st["kc"], "v_cache": st["vc"], "seq_lens": (base + st["accepted_lens"]).to(torch.int32)}


# ---------------------------------------------------------------- one pass
def _kept(st, name, make):
    """What a program makes once and keeps: the rotary handle, a workspace."""
    if name not in st:
        st[name] = make()
    return st[name]


def _own(st):
    import paged_kv_cache_mapping_gb300 as pkv
    c = st["case"]
    scale = CODE_SCALE if c.get("cache") == "e4m3" else 1.0
    if c["op"] == "rope":
        rope = _kept(st, "handle", lambda: pkv.pkv_rope_init(**st["rope"]))
        pkv.pkv_rope_append(st["q"], st["k"], st["v"], st["positions"], st["slots"], rope, st["kc"], st["vc"],
                            q_out=st["q_out"], k_scale=scale, v_scale=scale)
        return {"q": st["q_out"], "k_cache": st["kc"], "v_cache": st["vc"]}
    if c["op"] == "mask":
        return list(pkv.pkv_tree_mask(st["parents"], st["cu"], st["n"], st["max_q"]))
    if c["op"] == "commit":
        pkv.pkv_tree_commit(st["accepted"], st["accepted_lens"], st["cu"], st["n"], st["bt"], st["kc"], st["vc"],
                            new_seq_lens=st["new_n"])
        return {"k_cache": st["kc"], "v_cache": st["vc"], "seq_lens": st["new_n"]}
    ws = _kept(st, "ws", lambda: torch.empty(
        pkv.pkv_tree_attention_workspace_size(st["q"], st["bt"], st["kc"], st["max_q"]), dtype=torch.uint8, device="cuda"))
    return pkv.pkv_tree_attention(st["q"], st["cu"], st["n"], st["bt"], st["kc"], st["vc"], st["mask"], c["D"] ** -0.5,
                                  st["out"], k_scale=scale, v_scale=scale, max_q_len=st["max_q"], workspace=ws)


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "rope":
        return _plain_rope(st)
    if op == "mask":
        return list(_plain_mask(st["parents"], st["cu"], st["n"], st["T"], st["max_q"]))
    if op == "commit":
        return _plain_commit(st)
    return _plain_tree(st)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = 1 if case.get("cache") == "e4m3" else 2
    if case["op"] == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        return {"bytes": T * (4 * Hq * D + 2 * Hkv * D * (2 + es) + 8), "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    ctx, q = _lengths(case)
    T = sum(q)
    if case["op"] == "mask":
        return {"bytes": T * (4 + 4 + 4 * -(-max(q) // 32)) + 8 * case["B"], "flops": T}
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "commit":
        rows = case["B"] * (case["path"] + 1) / 2  # a path has 1 .. path nodes
        return {"bytes": int(4 * rows * Hkv * D * es) + 20 * case["B"], "flops": 0}
    n = [a + b for a, b in zip(ctx, q)]
    tables = 4 * sum(-(-m // case["bs"]) for m in n)
    rows = 4 * T * case["Hq"] * D
    return {"bytes": 2 * sum(n) * Hkv * D * es + rows + tables + 4 * T * -(-max(q) // 32),
            "flops": 4 * D * case["Hq"] * sum(a * b for a, b in zip(n, q))}


# ---------------------------------------------------------------- 64 bits
def _exact_rope(st):
    c, r = st["case"], st["rope"]
    rot, T = c["rot"], c["T"]
    f, m = _frequencies(rot, r["base"], r["scaling"], r.get("factor", 1.0), r.get("original_max_position", 0))
    turn = st["positions"].double()[:, None] * f
    z = m * torch.polar(torch.ones_like(turn), turn)[:, None, :]  # complex rotation of the pairs

    def rotated(x):
        x = x.double().clone()
        a = x[..., 0:rot:2] if c["interleaved"] else x[..., :rot // 2]
        b = x[..., 1:rot:2] if c["interleaved"] else x[..., rot // 2:rot]
        w = torch.complex(a.contiguous(), b.contiguous()) * z
        if c["interleaved"]:
            x[..., 0:rot:2], x[..., 1:rot:2] = w.real, w.imag
        else:
            x[..., :rot // 2], x[..., rot // 2:rot] = w.real, w.imag
        return x

    kc, vc = st["kc"].double(), st["vc"].double()
    s = 1.0 / CODE_SCALE if c["cache"] == "e4m3" else 1.0
    for cache, rows in ((kc, rotated(st["k"])), (vc, st["v"].double())):
        flat = cache.view(-1, c["Hkv"], c["D"])
        flat[st["slots"].long()] = (rows * s).clamp(-448, 448) if s != 1.0 else rows
    return {"q": rotated(st["q"]), "k_cache": kc, "v_cache": vc}


def _exact_tree(st):
    c = st["case"]
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["bs"]
    s = CODE_SCALE if c["cache"] == "e4m3" else 1.0
    cu, n = st["cu"].tolist(), st["n"].tolist()
    out = torch.zeros((cu[-1], Hq, D), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        m = cu[b + 1] - cu[b]
        blocks = st["bt"][b, :-(-n[b] // bs)].long()
        k, v = (x[blocks].reshape(-1, Hkv, D)[:n[b]].double() * s for x in (st["kc"], st["vc"]))
        words = st["mask"][cu[b]:cu[b + 1]].long()
        jj = torch.arange(m, device="cuda")
        seen = torch.ones((m, n[b]), dtype=torch.bool, device="cuda")
        seen[:, n[b] - m:] = (words[:, jj // 32] >> (jj % 32)) & 1 == 1
        for h in range(Hkv):
            q = st["q"][cu[b]:cu[b + 1], h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
            e = torch.einsum("igd,jd->igj", q, k[:, h]) * D ** -0.5
            e = e.masked_fill(~seen[:, None, :], -math.inf)
            p = torch.softmax(e, -1).nan_to_num(0.0)  # a row that sees nothing is zero
            out[cu[b]:cu[b + 1], h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = torch.einsum("igj,jd->igd", p, v[:, h])
    return out


def _exact_commit(st):
    c = st["case"]
    kc, vc = st["kc"].double(), st["vc"].double()
    cu, n, bt = st["cu"].tolist(), st["n"].tolist(), st["bt"].tolist()
    path, lens = st["accepted"].tolist(), st["accepted_lens"].tolist()
    for b in range(c["B"]):
        base = n[b] - (cu[b + 1] - cu[b])
        place = lambda p: (bt[b][p // c["bs"]], p % c["bs"])  # noqa: E731, B023
        for i in range(lens[b]):  # ascending: a row moves before its place is taken
            if path[b][i] != i:
                (x, y), (w, z) = place(base + i), place(base + path[b][i])
                kc[x, y] = kc[w, z]
                vc[x, y] = vc[w, z]
    return {"k_cache": kc, "v_cache": vc, "seq_lens": None}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "tree":
        return _exact_tree(st)
    if case["op"] == "commit":
        return _exact_commit(st)
    return None
