"""Many small weights behind one large one: a key whose score leads those of
thousands of others, with values of one sign against it, so that weights that
are lost or cut show in full instead of averaging out."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import tree_attention

pytestmark = pytest.mark.gpu

BS, KEYS = 64, 16384  # keys of a chunk in every case below


def bound(q, k, scale, top, n, kv):
    """Largest |error| of an fp32 output whose values are all +-1.  A weighted
    mean of values of size 1 whose weights are each off by a relative e moves
    by at most 2 e (numerator and sum).  e adds up
      - P.  e4m3 caches: one f16, half a step 2^-11, and 2^-25 for what is below
        f16's normal numbers, where the chunk's largest weight is at least 2^8: n
        keys lose at most n * 2^-33 of it.  bf16 caches: two parts, 2^-15;
      - the score: D = 128 fp32 additions of terms that sum to at most top,
        the exponent's argument and the exponential, 2^-22 (top + 2), and, e4m3,
        the query row in two codes, exact to 2^-18 of its largest element;
      - fp32 sums of n products, 16 at a time: (n / 16 + 16) * 2^-22."""
    e = 2.0 ** -11 + n * 2.0 ** -33 if kv == "e4m3" else 2.0 ** -15
    e += 128 * 2.0 ** -24 * top + 2.0 ** -22 * (top + 2)
    if kv == "e4m3":
        e += 2.0 ** -18 * scale * float(np.abs(q).max() * np.abs(k).sum(-1).max())
    return 2 * (e + (n / 16 + 16) * 2.0 ** -22)


def lead_case(kv, q_s, G, D, B, Hkv, ctx, nats, spread, seed):
    """B sequences over the same pages: key 5 of every chunk of KEYS leads by `nats`
    the others' mean, whose scores have a deviation of `spread` nats."""
    gen = torch.Generator().manual_seed(seed)
    n = ctx + q_s
    nb = -(-n // BS)
    scale, cs = D ** -0.5, 1.0 / 64
    q0 = torch.randn((Hkv, D), generator=gen).bfloat16().double()
    k = spread * torch.randn((nb * BS, Hkv, D), generator=gen, dtype=torch.float64)
    k[5:ctx:KEYS] = q0 * (nats / (scale * (q0 * q0).sum(1, keepdim=True)))
    v = torch.ones((nb * BS, Hkv, D), dtype=torch.float64)
    v[5:ctx:KEYS] = -1.0
    if kv == "e4m3":
        kc = (k / cs).clamp(-448, 448).float().to(torch.float8_e4m3fn)
        k_of, ks = kc.double() * cs, cs
        vc = v.float().to(torch.float8_e4m3fn)
    else:
        kc, vc, ks = k.bfloat16(), v.bfloat16(), 1.0
        k_of = kc.double()
    words = -(-q_s // 32)
    mask = np.zeros((q_s, words), np.uint32)
    for i in range(q_s):
        mask[i, i // 32] = 1 << (i % 32)
    rows = q0.repeat_interleave(G, 0).bfloat16()  # every node asks the same
    q = rows[None].expand(B * q_s, Hkv * G, D).contiguous()
    dev = dict(q=q.cuda(), cu=(torch.arange(B + 1, dtype=torch.int32) * q_s).cuda(),
               n=torch.full((B,), n, dtype=torch.int32).cuda(),
               bt=torch.arange(nb, dtype=torch.int32)[None].expand(B, nb).contiguous().cuda(),
               kc=kc.view(nb, BS, Hkv, D).cuda(), vc=vc.view(nb, BS, Hkv, D).cuda(),
               mask=torch.from_numpy(np.tile(mask.view(np.int32), (B, 1))).cuda())
    out = torch.full((B * q_s, Hkv * G, D), 7.0, device="cuda")
    pkv.pkv_tree_attention(dev["q"], dev["cu"], dev["n"], dev["bt"], dev["kc"], dev["vc"], dev["mask"], scale, out,
                           k_scale=ks, v_scale=1.0, max_q_len=q_s)
    assert pkv.pkv_device_errors() == 0
    kk, vv = k_of[:n].numpy(), v[:n].numpy()
    one = rows[::G].double().numpy()[None]  # a node's rows are alike, and so are the nodes but for their own key
    top, worst = 0.0, 0.0
    got = out.cpu().double().numpy().reshape(B, q_s, Hkv, G, D)
    for i in {0, q_s // 2, q_s - 1}:
        live = np.r_[0:ctx, ctx + i]
        want, t = tree_attention(one, kk[live], vv[live], np.ones((1, 1), np.int32), scale)
        top = max(top, t)
        worst = max(worst, float(np.abs(got[:, i] - want[0][None, :, None]).max()))
    tol = bound(one[0], kk, scale, top, min(n, KEYS + q_s), kv)
    assert worst <= tol, f"max err {worst:.3e}, bound {tol:.3e}"
    assert tol < 0.01


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("nats", [6.0, 8.0, 9.0, 10.0, 11.0, 12.5])
@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
def test_a_leading_key_over_one_long_chunk(kv, nats, spread):
    """More than 512 nodes: a sequence is one chunk."""
    lead_case(kv, 516, 1, 64, 1, 1, KEYS - 516, nats, spread, 7)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_s,G", [(4, 4), (8, 4), (16, 4), (20, 4)])
@pytest.mark.parametrize("nats", [8.0, 10.5, 12.0])
@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
def test_a_leading_key_in_every_chunk(kv, nats, q_s, G, D):
    """152 (sequence, KV head) units of 131,072 keys: eight chunks each, every tile width."""
    lead_case(kv, q_s, G, D, 76, 2, 8 * KEYS - q_s, nats, 1.0, 8)
