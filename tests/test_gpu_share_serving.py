"""A serving loop whose tables, lengths and free list live on the GPU: requests
behind a shared prompt are admitted, grow, lose drafted tokens and end, by
pkv_step_tables, pkv_append, pkv_shared_prefixes and pkv_shared_attention alone;
eagerly and as one captured graph.  Every row is checked against 64-bit
attention over each request's own logical keys."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.spec_ref import attention_tolerance, tree_attention

pytestmark = pytest.mark.gpu
BS, W, HQ, HKV, D, B, T = 16, 24, 8, 2, 64, 7, 160
PREFIX = 5 * BS  # of requests 0 .. 4; the others have none
SHARED = [5] * 5 + [0, 0]


class Server:
    def __init__(self, kv, seed):
        g = torch.Generator().manual_seed(seed)
        self.r, self.g, self.kv = random.Random(seed), g, kv
        self.scale = D ** -0.5
        self.ks, self.vs = (0.011, 0.013) if kv == "e4m3" else (1.0, 1.0)
        pool = 120
        cdt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
        self.kc, self.vc = (torch.zeros((pool, BS, HKV, D), device="cuda").to(cdt) for _ in range(2))
        perm = torch.randperm(pool, generator=g).to(torch.int32)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bt = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.bt[:5, :5] = perm[:5].cuda()  # the shared prompt's blocks are in everybody's table
        self.free = torch.cat([perm[5:], torch.full((5,), -1, dtype=torch.int32)]).cuda()
        self.count, self.shared = i32([pool - 5]), i32(SHARED)
        self.old, self.new, self.cu = i32([0] * B), i32([0] * B), i32([0] * (B + 1))
        self.slots, self.groups = i32([0] * T), torch.zeros((B, 3), dtype=torch.int32, device="cuda")
        self.q = torch.zeros((T, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.k, self.v = (torch.zeros((T, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.out = torch.full((T, HQ, D), 7.0, device="cuda")
        self.ws = torch.empty(pkv.pkv_shared_attention_workspace_size(self.q, self.bt, self.kc), dtype=torch.uint8, device="cuda")
        # the shared prompt's keys and values, and the logical ones of every request
        k, v = self.rows(PREFIX), self.rows(PREFIX)
        at = (self.bt[0, :5].long()[:, None] * BS + torch.arange(BS, device="cuda")[None]).flatten().to(torch.int32)
        pkv.pkv_append(k.cuda(), v.cuda(), at, self.kc, self.vc, self.ks, self.vs)
        self.logical = [(self.seen(k, self.ks), self.seen(v, self.vs)) if s < 5 else (np.zeros((0, HKV, D)),) * 2 for s in range(B)]
        self.len = [PREFIX if s < 5 else 0 for s in range(B)]

    def rows(self, n):
        return torch.randn((n, HKV, D), generator=self.g).to(torch.bfloat16)

    def seen(self, x, s):
        """What the cache holds of rows x."""
        if self.kv == "bf16":
            return x.double().numpy()
        codes = (x.float() * torch.tensor(1.0 / np.float32(s), dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes.double().numpy() * s

    def step(self):
        pkv.pkv_step_tables(self.old, self.new, self.bt, BS, self.free, self.count, self.cu, self.slots, shared_blocks=self.shared)
        pkv.pkv_append(self.k, self.v, self.slots, self.kc, self.vc, self.ks, self.vs)
        pkv.pkv_shared_prefixes(self.cu, self.new, self.bt, BS, min_tokens=2 * BS, groups=self.groups)
        pkv.pkv_shared_attention(self.q, self.cu, self.new, self.bt, self.groups, self.kc, self.vc, self.scale, self.out,
                                 k_scale=self.ks, v_scale=self.vs, workspace=self.ws)

    def next(self):
        """The requests' next lengths: decodes, prompts, rejected drafts, ends."""
        least = [PREFIX if s < 5 else 0 for s in range(B)]
        new = []
        for s, n in enumerate(self.len):
            u = self.r.random()
            if n == least[s]:
                new.append(n + self.r.randint(1, 20))
            elif u < 0.15 or n > (W - 2) * BS:
                new.append(least[s])  # done: its own blocks go back
            elif u < 0.3:
                new.append(max(least[s], n - self.r.randint(1, 5)))
            else:
                new.append(n + self.r.choice([1, 1, 1, 4]))
        return new

    def load(self, new):
        rows = [max(0, b - a) for a, b in zip(self.len, new)]
        n = sum(rows)
        q = (1.5 * torch.randn((n, HQ, D), generator=self.g)).to(torch.bfloat16)
        k, v = self.rows(n), self.rows(n)
        for dst, src in ((self.q, q), (self.k, k), (self.v, v)):
            dst[:n] = src.cuda()
        self.old.copy_(torch.tensor(self.len, dtype=torch.int32))
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.out.fill_(7.0)
        at = 0
        for s in range(B):
            lk, lv = self.logical[s]
            self.logical[s] = tuple(np.concatenate([x[:min(self.len[s], new[s])], self.seen(y[at:at + rows[s]], z)])
                                    for x, y, z in ((lk, k, self.ks), (lv, v, self.vs)))
            at += rows[s]
        self.len = new
        return q, rows

    def check(self, q, rows):
        assert pkv.pkv_device_errors() == 0
        got, at = self.out.cpu().double().numpy(), 0
        blocks = 5 + sum(-(-n // BS) - sh for n, sh in zip(self.len, SHARED))
        assert int(self.count) == self.kc.shape[0] - blocks  # none lost, none given twice
        used = [int(self.bt[s, j]) for s in range(B) for j in range(SHARED[s], -(-self.len[s] // BS))] + self.bt[0, :5].tolist()
        assert len(set(used)) == blocks and not set(used) & set(self.free[:int(self.count)].tolist())
        for s in range(B):
            k, v = self.logical[s]
            assert len(k) == self.len[s]
            if rows[s]:
                words = -(-rows[s] // 32)
                mask = np.zeros((rows[s], words), np.uint32)
                for i in range(rows[s]):
                    for j in range(i + 1):
                        mask[i, j // 32] |= np.uint32(1 << (j % 32))
                want, top = tree_attention(q[at:at + rows[s]].double().numpy(), k, v, mask.view(np.int32), self.scale)
                tol = attention_tolerance(float(np.abs(v).max()), top, len(k), self.kv)
                assert np.abs(got[at:at + rows[s]] - want).max() <= tol, s
            at += rows[s]
        assert (self.out[at:] == 7.0).all()
        return self.groups.tolist()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(kv, captured):
    s = Server(kv, 7 + captured)
    run = s.step
    if captured:
        s.step()  # one-time set-up: no request grows
        assert pkv.pkv_device_errors() == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        run = graph.replay
    shared = 0
    for _ in range(14):
        work = s.load(s.next())
        run()
        shared += sum(p > 0 for _, _, p in s.check(*work))
    assert shared > 14  # the prefix was shared by several requests in most steps
