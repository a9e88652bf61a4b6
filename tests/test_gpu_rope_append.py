"""pkv_rope_append against a 64-bit rotation: layouts, partial rotation, the
long-context scalings, far and negative positions, strided and in-place rows,
skipped and out-of-range slots, every dtype pair."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import HALF_STEP, frequencies, rotate

pytestmark = pytest.mark.gpu

CDT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def make(T, Hq, Hkv, D, src, cache, max_pos, seed, pos_dtype=torch.int32, slot_dtype=torch.int32, bs=16):
    g = torch.Generator().manual_seed(seed)
    dt = CDT[src]
    qkv = torch.randn((T, (Hq + 2 * Hkv), D), generator=g).to(dt)
    pos = torch.randint(0, max_pos, (T,), generator=g).to(pos_dtype)
    nb = -(-T // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T].to(slot_dtype)
    kc = torch.randn((nb, bs, Hkv, D), generator=g).to(CDT[cache])
    vc = torch.randn((nb, bs, Hkv, D), generator=g).to(CDT[cache])
    return qkv, pos, slots, kc, vc


def angle_tolerance(x, amp, max_pos):
    """|error| of the fp32 rotation: the turn as a float (2^-25 half turns, pi
    2^-25 rad), the fixed-point turns (pos * 2^-53 relative to the frequency,
    as the 64-bit reference's own angle), sincospif (2 ulp, 2^-22) and three
    fp32 roundings of products of at most |a| + |b|."""
    return 2 * float(x.abs().max()) * amp * (3.2 * 2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -24 + 8 * max_pos * 2.0 ** -53)


def close(got, want, dt, tol):
    got, want = got.double().numpy(), np.asarray(want)
    assert np.isfinite(got).all()
    bound = tol + HALF_STEP[dt] * np.abs(want) * (1 + 2.0 ** -6) if dt != torch.float32 else tol
    err = np.abs(got - want)
    assert (err <= bound).all(), f"max err {err.max():.3e}"


def check(T=37, Hq=8, Hkv=2, D=128, rot=128, interleaved=False, scaling="none", src="bf16", cache="bf16",
          max_pos=5000, base=10000.0, factor=1.0, L=0.0, seed=1, in_place=False, pos=None, **kw):
    qkv, p, slots, kc, vc = make(T, Hq, Hkv, D, src, cache, max_pos, seed, **kw)
    p = p if pos is None else pos
    ks, vs = (0.011, 0.013) if cache == "e4m3" else (1.0, 1.0)
    f, amp = frequencies(rot, base, scaling, factor, L)
    dev = qkv.cuda()  # q, k, v are views of one fused buffer
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    gk, gv = kc.cuda(), vc.cuda()
    rope = pkv.pkv_rope_init(rot, base, interleaved, scaling, factor, L)
    out = pkv.pkv_rope_append(q, k, v, p.cuda(), slots.cuda(), rope, gk, gv, q_out=q if in_place else None, k_scale=ks,
                              v_scale=vs)
    torch.cuda.synchronize()
    assert pkv.pkv_device_errors() == 0
    x = qkv.double().numpy()
    far = int(p.abs().max())
    tol = angle_tolerance(qkv, amp, far)
    close(out.cpu(), rotate(x[:, :Hq], p.numpy(), f, amp, rot, interleaved), CDT[src], tol)
    want_k, want_v = kc.double().numpy().copy(), vc.double().numpy().copy()
    rk = rotate(x[:, Hq:Hq + Hkv], p.numpy(), f, amp, rot, interleaved) / ks
    rv = x[:, Hq + Hkv:] / vs
    sl = slots.long().numpy()
    for want, rows in ((want_k, rk), (want_v, rv)):
        want.reshape(-1, Hkv, D)[sl] = np.clip(rows, -448, 448) if cache == "e4m3" else rows
    extra = 2.0 ** -10 if cache == "e4m3" else 0.0  # half the smallest e4m3 step
    close(gk.cpu(), want_k, CDT[cache], tol / ks + extra)
    close(gv.cpu(), want_v, CDT[cache], extra + 2.0 ** -20)
    # v rows are those of pkv_append, bit for bit
    gk2, gv2 = kc.cuda(), vc.cuda()
    pkv.pkv_append(k, v, slots.cuda(), gk2, gv2, ks, vs)
    assert torch.equal(gv.view(torch.uint8), gv2.view(torch.uint8))


@pytest.mark.parametrize("src,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dtypes_and_layouts(src, cache, interleaved):
    check(src=src, cache=cache, interleaved=interleaved, rot=64)


@pytest.mark.parametrize("T", [1, 2, 151, 700])
def test_token_counts(T):
    check(T=T, Hq=32, Hkv=8)


@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (64, 2), (64, 48), (128, 96), (256, 256), (8, 8), (72, 40),
                                   (128, 6), (128, 126), (40, 22)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_dims_and_partial_rotation(D, rot, interleaved):
    check(T=5, Hq=6, Hkv=3, D=D, rot=rot, interleaved=interleaved)
    check(T=5, Hq=3, Hkv=1, D=D, rot=rot, interleaved=interleaved, src="f32", cache="f32", seed=2)


@pytest.mark.parametrize("scaling,factor,L", [("linear", 4.0, 0.0), ("ntk", 8.0, 0.0), ("by_parts", 16.0, 4096.0),
                                              ("smooth", 8.0, 8192.0)])
def test_scalings(scaling, factor, L):
    check(scaling=scaling, factor=factor, L=L, base=500000.0, max_pos=131072)
    check(scaling=scaling, factor=factor, L=L, rot=32, src="f32", cache="f32", max_pos=131072, interleaved=True)


def test_far_and_negative_positions():
    far = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 1000003], dtype=torch.int32)
    check(T=7, src="f32", cache="f32", pos=far, max_pos=2 ** 31)
    check(T=7, src="f32", cache="f32", pos=far.long(), max_pos=2 ** 31, slot_dtype=torch.int64)
    # far beyond what a 64-bit angle holds: position p + 2^40 turns like the product of the two rotations
    rope = pkv.pkv_rope_init(64, 10000.0)
    from fractions import Fraction
    turns = [Fraction(rope.turns[i], 2 ** 64) for i in range(32)]
    pos = 2 ** 40 + 12345
    x = torch.randn((1, 1, 64), generator=torch.Generator().manual_seed(5))
    kc = torch.zeros((1, 1, 1, 64)).cuda()
    vc = kc.clone()
    got = pkv.pkv_rope_append(x.cuda(), x.cuda(), x.cuda(), torch.tensor([pos]).cuda(), torch.tensor([0]).cuda(), rope, kc,
                              vc).cpu().double().numpy()
    ang = np.array([float((pos * t) % 1) * 2 * np.pi for t in turns])
    want = rotate(x.double().numpy(), [1.0], ang, 1.0, 64, False)
    assert np.abs(got - want).max() <= angle_tolerance(x, 1.0, 1)


def test_in_place_and_wide_indices():
    check(T=33, in_place=True)
    check(T=33, in_place=True, interleaved=True, rot=34, pos_dtype=torch.int64, slot_dtype=torch.int64)


def test_skipped_and_out_of_range_slots():
    T, Hq, Hkv, D = 9, 4, 2, 64
    qkv, p, slots, kc, vc = make(T, Hq, Hkv, D, "bf16", "bf16", 100, 3)
    n = kc.shape[0] * kc.shape[1]
    slots[2], slots[5] = -1, n  # skipped; out of range: skipped and recorded
    dev, gk, gv = qkv.cuda(), kc.cuda(), vc.cuda()
    rope = pkv.pkv_rope_init(D)
    out = pkv.pkv_rope_append(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], p.cuda(), slots.cuda(), rope, gk, gv)
    assert pkv.pkv_device_errors() == 1
    f, amp = frequencies(D, 10000.0)
    close(out.cpu(), rotate(qkv.double().numpy()[:, :Hq], p.numpy(), f, amp, D, False), torch.bfloat16,
          angle_tolerance(qkv, 1.0, 100))
    kept = torch.ones(n, dtype=torch.bool)
    kept[[int(s) for i, s in enumerate(slots) if i not in (2, 5)]] = False
    assert torch.equal(gk.cpu().view(n, Hkv, D)[kept], kc.view(n, Hkv, D)[kept])
    assert torch.equal(gv.cpu().view(n, Hkv, D)[kept], vc.view(n, Hkv, D)[kept])


def test_graph_replay_takes_new_values():
    T, Hq, Hkv, D = 21, 8, 2, 128
    qkv, p, slots, kc, vc = make(T, Hq, Hkv, D, "bf16", "bf16", 4000, 6)
    dev, pos, sl, gk, gv = qkv.cuda(), p.cuda(), slots.cuda(), kc.cuda(), vc.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    rope = pkv.pkv_rope_init(D)
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_rope_append(q, k, v, pos, sl, rope, gk, gv, q_out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_rope_append(q, k, v, pos, sl, rope, gk, gv, q_out=out)
    pos.add_(77)
    dev.mul_(0.5)
    g.replay()
    got = out.clone()
    again = pkv.pkv_rope_append(q, k, v, pos, sl, rope, gk.clone(), gv.clone())
    torch.cuda.synchronize()
    assert torch.equal(got, again)
