"""The serving loop where only the first request's table still has the shared
prompt's blocks when attention runs: every row comes out right when, and only when, the prompt is read
once for all of them, in both cache formats, eagerly and captured."""
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.test_gpu_share_serving import BS, HQ, PREFIX, Server

pytestmark = pytest.mark.gpu


class OnePrompt(Server):
    def __init__(self, kv, seed):
        super().__init__(kv, seed)
        self.seen_by = self.bt.clone()
        # other blocks that the cache has, in place of the prompt's
        self.others = (torch.arange(4 * 5, dtype=torch.int32, device="cuda").view(4, 5) * 7 + 3) % self.kc.shape[0]

    def step(self):
        pkv.pkv_step_tables(self.old, self.new, self.bt, BS, self.free, self.count, self.cu, self.slots, shared_blocks=self.shared)
        pkv.pkv_append(self.k, self.v, self.slots, self.kc, self.vc, self.ks, self.vs)
        pkv.pkv_shared_prefixes(self.cu, self.new, self.bt, BS, min_tokens=2 * BS, groups=self.groups)
        self.seen_by.copy_(self.bt)
        self.seen_by[1:5, :5] = self.others
        pkv.pkv_shared_attention(self.q, self.cu, self.new, self.seen_by, self.groups, self.kc, self.vc, self.scale, self.out,
                                 k_scale=self.ks, v_scale=self.vs, workspace=self.ws)

    def next(self):
        """Few rows each, so that the requests behind the prompt share it; one of them may end."""
        new = [n + self.r.choice([1, 1, 2, 3]) for n in self.len]
        s = self.r.randrange(7)
        if self.len[s] > (PREFIX if s < 5 else 0):
            new[s] = PREFIX if s < 5 else 0
        return new


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_the_prompt_is_read_for_all(kv, captured):
    s = OnePrompt(kv, 17 + captured)
    assert HQ == 8
    run = s.step
    if captured:
        s.step()  # one-time set-up: no request grows
        assert pkv.pkv_device_errors() == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        run = graph.replay
    for _ in range(12):
        work = s.load(s.next())
        run()
        assert s.check(*work)[:5] == [[0, 5, PREFIX]] * 5
