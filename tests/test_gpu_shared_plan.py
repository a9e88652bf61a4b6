"""Calls that look through the groups first (buffers of many more rows than the
requests have, bounds unknown): what is recorded and left as it is, graphs that
share a workspace, another stream, and lengths that make no sense."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.share_ref import SharedBatch
from tests.test_gpu_shared import GROUPS, Dev, close
from tests.test_gpu_shared_sharing import padded

pytestmark = pytest.mark.gpu
T = 1500


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(GROUPS))
def test_bad_groups_are_recorded(name, kv):
    b = SharedBatch([(4, 64), (1, 0), (2, 32)], [40, 3, 17, 1, 30, 8, 1], [1, 2, 1, 1, 3, 1, 1], 4, 2, 64, 16, kv, seed=91)
    d = Dev(b)
    GROUPS[name](d.groups)
    out = padded(d, T)
    d.run(max_q=0, max_group=0)
    assert pkv.pkv_device_errors() == 4
    got = out.cpu()
    assert (got[b.T:] == 7.0).all()
    got = got[:b.T]
    close(b, got, slice(int(b.cu[4]), None))
    for s in range(4):  # left as they were, or (a request whose own numbers hold) right
        rows = slice(int(b.cu[s]), int(b.cu[s + 1]))
        if not (got[rows] == 7.0).all():
            assert name in ("first with another prefix", "first without a prefix") and s == 0
            close(b, got, rows)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_requests_beyond_their_bounds_and_tables(kv):
    b = SharedBatch([(5, 64), (3, 32)], [40, 3, 17, 1, 30, 8, 1, 0], [1, 2, 1, 9, 3, 1, 1, 2], 4, 2, 64, 16, kv, seed=92)
    for s, change, bounds in ((3, lambda d: None, (8, 0)), (1, lambda d: d.n.__setitem__(1, 60), (0, 0)),
                              (6, lambda d: d.n.__setitem__(6, 1 << 30), (0, 0)), (0, lambda d: d.n.__setitem__(0, -1), (0, 0))):
        d = Dev(b)
        change(d)
        out = padded(d, T)
        d.run(*bounds)
        assert pkv.pkv_device_errors() == 4
        for r in range(b.B):
            rows = slice(int(b.cu[r]), int(b.cu[r + 1]))
            if r == s:
                assert (out[rows] == 7.0).all()
            else:
                close(b, out[:b.T], rows)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_lengths_that_make_no_sense_are_recorded(kv):
    b = SharedBatch([(40, 64)], [5] * 40, [1 + s % 3 for s in range(40)], 4, 2, 64, 16, kv, seed=93)
    r = np.random.default_rng(93)
    for values in ((0, b.T), (0, T), (-5, T + 9), (-2 ** 31, 2 ** 31 - 1)):
        for _ in range(4):
            d = Dev(b)
            at = r.integers(0, 41, 12)
            d.cu[torch.from_numpy(at).cuda()] = torch.from_numpy(r.integers(*values, 12, dtype=np.int32)).cuda()
            padded(d, T)
            d.run(max_q=0, max_group=0)
            assert pkv.pkv_device_errors() == 4
    # every other request begins at row 0 again: in all they claim more rows than there are
    d = Dev(b)
    d.cu[0::2] = 0
    d.cu[1::2] = 100
    d.cu[40] = 100
    d.n.fill_(64 + 110)
    d.bt = torch.zeros((40, 20), dtype=torch.int32, device="cuda")
    out = padded(d, T)
    d.run(max_q=0, max_group=0)
    assert pkv.pkv_device_errors() == 4
    assert (out[100:] == 7.0).all()


def test_graphs_that_share_a_workspace_follow_their_inputs():
    b = SharedBatch([(6, 256), (2, 64)], [50, 3, 0, 200, 17, 1, 90, 4], [1] * 7 + [60], 8, 2, 64, 16, "bf16", seed=94)
    d, e = Dev(b), Dev(b)
    outs = [padded(x, T) for x in (d, e)]
    d.run(0, 0)  # one-time set-up
    ws = torch.empty(pkv.pkv_shared_attention_workspace_size(d.q, d.bt, d.kc), dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (d, e):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(0, 0, workspace=ws)
        graphs.append(g)
    e.q[:b.T].neg_()
    ws.fill_(255)
    for o in outs:
        o.fill_(7.0)
    for g in graphs + graphs:
        g.replay()
    assert pkv.pkv_device_errors() == 0
    close(b, outs[0][:b.T])
    want = e.run(0, 0, out=torch.full_like(outs[1], 7.0))
    assert torch.equal(outs[1], want)
    # nothing shared, then other groups: nothing of the first ones is kept
    for groups in (torch.zeros_like(d.groups), pkv.pkv_shared_prefixes(d.cu, d.n, d.bt, 16, min_tokens=16)):
        d.groups.copy_(groups)
        outs[0].fill_(7.0)
        graphs[0].replay()
        assert pkv.pkv_device_errors() == 0
        close(b, outs[0][:b.T])


def test_two_calls_at_once():
    shape = ([(8, 512)], [50] * 8, [1] * 7 + [40], 8, 2, 128, 16)
    a, b = Dev(SharedBatch(*shape, "bf16", seed=95)), Dev(SharedBatch(*shape, "e4m3", seed=96))
    oa, ob = padded(a, T), padded(b, T)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run(0, 0)
        with torch.cuda.stream(s2):
            b.run(0, 0)
    torch.cuda.synchronize()
    assert pkv.pkv_device_errors() == 0
    close(a.b, oa[:a.b.T])
    close(b.b, ob[:b.b.T])
