"""Plain 64-bit references of the speculative decoding operators, and the
inputs of their tests.  numpy and torch on the CPU only; no library call."""
import math

import numpy as np
import torch

from tests.helpers import random_tables

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


# ---------------------------------------------------------------- rotary positions
def frequencies(rot, base, scaling="none", factor=1.0, L=0.0):
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    amp = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "ntk":
        b = base * factor ** (rot / (rot - 2)) if rot > 2 else base
        f = [b ** (-2.0 * i / rot) for i in range(rot // 2)]
    elif scaling == "by_parts":
        pair = lambda turns: rot * math.log(L / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        out = []
        for i, x in enumerate(f):
            r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            out.append(x * (1 - r) + x / factor * r)
        f, amp = out, 0.1 * math.log(factor) + 1.0
    elif scaling == "smooth":
        out = []
        for x in f:
            w = min(max((L * x / (2 * math.pi) - 1) / 3, 0.0), 1.0)
            out.append(w * x + (1 - w) * x / factor)
        f = out
    return np.array(f), amp


def rotate(x, positions, f, amp, rot, interleaved):
    """x [T, H, D] float64 -> rotated, float64."""
    x = np.array(x, np.float64)
    ang = np.asarray(positions, np.float64)[:, None] * f[None, :]
    c, s = amp * np.cos(ang)[:, None, :], amp * np.sin(ang)[:, None, :]
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = a * s + b * c
    return x


# ---------------------------------------------------------------- trees
def tree_mask(parents, q_lens, seq_lens, words):
    mask = np.zeros((len(parents), words), np.uint32)
    pos = np.zeros(len(parents), np.int32)
    at = 0
    for q, n in zip(q_lens, seq_lens):
        for i in range(q):
            j, depth = i, 0
            while True:
                mask[at + i, j // 32] |= np.uint32(1 << (j % 32))
                if parents[at + j] < 0:
                    break
                j, depth = parents[at + j], depth + 1
            pos[at + i] = n - q + depth
        at += q
    return mask.view(np.int32), pos


def tree_attention(q, k_rows, v_rows, mask, scale):
    """One sequence: q [m, Hq, D], k_rows / v_rows [n, Hkv, D] (float64),
    mask [m, W] int32.  Returns (out [m, Hq, D], bound of scale * |q|.|k|)."""
    m, Hq, D = q.shape
    n, Hkv, _ = k_rows.shape
    G = Hq // Hkv
    ctx = n - m
    seen = np.ones((m, n), bool)
    w = mask.view(np.uint32)
    for j in range(m):
        seen[:, ctx + j] = (w[:, j // 32] >> np.uint32(j % 32)) & 1
    out = np.zeros((m, Hq, D))
    top = 0.0
    for h in range(Hq):
        g = h // G
        if n == 0:
            continue
        x = np.where(seen, scale * (q[:, h] @ np.where(np.isfinite(k_rows[:, g]), k_rows[:, g], 0.0).T), -np.inf)
        bad = ~np.isfinite(k_rows[:, g]).all(1)
        x[:, bad] = np.where(seen[:, bad], np.nan, -np.inf)
        fin = np.where(np.isfinite(k_rows[:, g]), np.abs(k_rows[:, g]), 0.0)
        top = max(top, float((abs(scale) * (np.abs(q[:, h]) @ fin.T)).max()))
        mx = x.max(1, keepdims=True)
        p = np.where(seen, np.exp(x - np.where(np.isfinite(mx), mx, 0.0)), 0.0)
        s = p.sum(1)
        for i in range(m):
            if s[i] == 0:
                continue
            live = seen[i]
            out[i, h] = (p[i, live] @ v_rows[live, g]) / s[i]
    return out, top


def attention_tolerance(vmax, top, n, kv):
    """Largest |error| of an fp32 output against 64 bits: a weighted mean of
    values of size vmax whose weights are each off by a relative e moves by
    at most 2 e vmax (numerator and sum).  e adds up
      - the score's error, D = 128 fp32 additions of terms that sum to at most
        top in absolute value (scaled): 128 * 2^-24 * top, and the rounding of
        the exponent's argument and the exponential itself: 2^-22 (top + 2);
      - P in two parts: bf16 hi + lo, 2^-16; e4m3 hi + lo, 2^-8 (half a step of
        half a step, 2^-4 * 2^-4) and 2^-17 of the row's largest weight for the
        smallest codes; one part in fp32: none;
      - the fp32 sums over n keys, at most n * 2^-24 relative."""
    part = {"f32": 0.0, "bf16": 2.0 ** -15, "e4m3": 2.0 ** -8 + n * 2.0 ** -17 / max(1.0, n ** 0.5)}[kv]
    e = 128 * 2.0 ** -24 * top + 2.0 ** -22 * (top + 2) + part + n * 2.0 ** -24
    return 2 * e * vmax


class Batch:
    """A ragged batch of trees over a shuffled paged cache (CPU tensors)."""

    def __init__(self, ctx, q_lens, Hq, Hkv, D, bs, kv, seed, parents=None, slack=3, width=None, mask_words=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.ctx, self.q_lens = list(ctx), list(q_lens)
        self.n = [a + b for a, b in zip(self.ctx, self.q_lens)]
        self.B, self.T, self.Hq, self.Hkv, self.D, self.bs, self.kv = len(self.n), sum(self.q_lens), Hq, Hkv, D, bs, kv
        self.max_q = max(self.q_lens + [1])
        self.words = mask_words or -(-self.max_q // 32)
        self.cu = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        nb = sum(-(-x // bs) for x in self.n) + slack
        self.nb = nb
        self.tables = random_tables(rng, self.n, bs, nb, width=width)
        self.scale = D ** -0.5
        self.src = torch.float32 if kv == "f32" else torch.bfloat16
        self.q = (1.5 * torch.randn((self.T, Hq, D), generator=gen)).to(self.src)
        self.k_scale, self.v_scale = (0.011, 0.013) if kv == "e4m3" else (1.0, 1.0)
        cdt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kv]
        mk = lambda s: (torch.randn((nb, bs, Hkv, D), generator=gen) / s).clamp(-448 if kv == "e4m3" else -1e9, 448 if kv == "e4m3" else 1e9).to(cdt)  # noqa: E731,E501
        self.kc, self.vc = mk(self.k_scale), mk(self.v_scale)
        if parents is None:
            parents = []
            for q in self.q_lens:
                parents += [int(rng.integers(-1, i)) if i else -1 for i in range(q)]
        self.parents = np.array(parents, np.int32)
        self.mask, self.pos = tree_mask(self.parents, self.q_lens, self.n, self.words)

    def slots(self, s):
        """Flat slots of sequence s's positions."""
        p = np.arange(self.n[s])
        return self.tables[s][p // self.bs].astype(np.int64) * self.bs + p % self.bs if self.n[s] else p

    def rows(self, s):
        sl = torch.from_numpy(self.slots(s))
        k = self.kc.double().view(-1, self.Hkv, self.D)[sl].numpy() * self.k_scale
        v = self.vc.double().view(-1, self.Hkv, self.D)[sl].numpy() * self.v_scale
        return k, v

    def reference(self):
        out = np.zeros((self.T, self.Hq, self.D))
        top, vmax = 0.0, 0.0
        for s in range(self.B):
            a, b = self.cu[s], self.cu[s + 1]
            if a == b:
                continue
            k, v = self.rows(s)
            out[a:b], t = tree_attention(self.q[a:b].double().numpy(), k, v, self.mask[a:b], self.scale)
            top = max(top, t)
            fin = np.abs(v[np.isfinite(v)])
            vmax = max(vmax, float(fin.max()) if fin.size else 0.0)
        return out, attention_tolerance(vmax, top, max(self.n), self.kv)
