"""Shared attention in 64 bits with a bound on the error of each element of the
output, from that row's own keys.  numpy and torch on the CPU only."""
import numpy as np

# A call cuts a request's keys into chunks of at most so many where it has more, and joins at most so many of them.
CHUNK, CHUNKS = 8192, 128


def relative(b, n, top, spread):
    """How far the weight of a key, or a sum of n of them, may be off, relative to it.

    Scores: D fp32 additions of exact products, a whole step each (2^-23), of terms that sum to `top` in absolute
    value; the scale's and the exponent's rounding, and the exponential: 2^-21 (top + 2).  On e4m3 caches a query row is
    two e4m3 codes for each element, scaled so that the largest is in 2^7 .. 2^8: the first is off by at most half a
    step, eight units of the bf16 element's last place, which the second holds exactly unless that place is below the
    codes' smallest number 2^-9; then half of that, 2^-17 of the largest element.
    Weights in the product with V: bf16 twice, each cut after 8 bits, 2^-15; on e4m3 caches f16, 2^-11, and half of
    its smallest number, 2^-33 of the row's largest weight, for each key.
    Sums: the products of 16 keys at a time, twice for two parts, over a chunk, with an error of at most 2^-22 of the
    sum of absolute values in each step (17 terms, cut where the largest ends); the sums of weights and of at most
    CHUNKS chunks: 2^-16; the chunks' weights: 2^-21 (top + 16)."""
    scores = b.D * 2.0 ** -23 * top + 2.0 ** -21 * (top + 2) + (2.0 ** -17 * spread if b.kv == "e4m3" else 0.0)
    part = {"bf16": 2.0 ** -15, "e4m3": 2.0 ** -11 + n * 2.0 ** -33, "f32": 0.0}[b.kv]
    steps = {"bf16": 2, "e4m3": 1, "f32": 16}[b.kv] * (min(n, CHUNK if b.kv != "f32" else n) / 16 + 8)
    return scores + part + steps * 2.0 ** -22 + 2.0 ** -16 + 2.0 ** -21 * (top + 16)


def reference(b, *lost):
    """(out, bound) [T, Hq, D].  A relative error e of every weight and of their sum moves an element by at most
    2 e sum w |v|.  For each of `lost`, a mask of the keys of request s (of n) that a wrong answer leaves out, also that
    answer."""
    outs, bound = np.zeros((1 + len(lost), b.T, b.Hq, b.D)), np.zeros((b.T, b.Hq, b.D))
    G = b.Hq // b.Hkv
    for s in range(b.B):
        keys, values = b.rows(s)
        gone = [f(s, b.n[s]) for f in lost]
        for g in range(b.Hkv):
            k, v = np.ascontiguousarray(keys[:, g]), np.ascontiguousarray(values[:, g])
            size, total = np.abs(k), np.abs(k).sum(1)
            for i in range(b.q_lens[s]):
                t, n = int(b.cu[s]) + i, b.ctx[s] + i + 1
                for h in range(g * G, (g + 1) * G):
                    q = b.q[t, h].double().numpy()
                    x = b.scale * (k[:n] @ q)
                    w = np.exp(x - x.max())
                    top, spread = abs(b.scale) * (size[:n] @ np.abs(q)).max(), abs(b.scale) * np.abs(q).max() * total[:n].max()
                    outs[0, t, h] = (w @ v[:n]) / w.sum()
                    bound[t, h] = 2 * relative(b, n, top, spread) * (w @ np.abs(v[:n])) / w.sum()
                    for o, m in zip(outs[1:], gone):
                        kept = np.where(m[:n], 0.0, w)
                        o[t, h] = (kept @ v[:n]) / kept.sum()
    return (outs[0], bound, *outs[1:])


LONG = {  # groups, own context, new tokens, Hq, Hkv, D, bs
    "long prefix and long requests": ([(3, 40000)], [9000, 1, 20000], [1, 2, 1], 4, 2, 64, 16),
    "one long request among short ones": ([(12, 128)], [1] * 11 + [30000], [1] * 12, 2, 2, 64, 16),
    "prefixes of many chunks": ([(5, 20480), (3, 8192)], [0, 700, 3, 1500, 64, 9, 2048, 0], [1, 2, 1, 1, 3, 1, 1, 1], 8, 2, 128, 16),
    "many rows behind a long prefix": ([(30, 6144)], [17 * s for s in range(30)], [1, 2, 1] * 10, 4, 1, 64, 32),
    "prompts behind a long prefix": ([(4, 4096)], [0, 300, 77, 1024], [40, 33, 20, 36], 4, 1, 64, 16),
    "a prompt and decodes": ([(10, 8192)], [5 * s for s in range(10)], [1, 1, 1, 150, 1, 1, 1, 1, 1, 1], 4, 1, 64, 16),
}
