"""The bound on each element of shared attention is one that a wrong answer does not pass (no GPU)."""
import numpy as np
import pytest

from tests.share_ref import SharedBatch
from tests.share_rows import LONG, reference


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", ["long prefix and long requests", "one long request among short ones", "prefixes of many chunks"])
def test_wrong_answers_do_not_pass(name, kv):
    b = SharedBatch(*LONG[name], kv=kv, seed=81)
    prefix = [p for _, _, p in b.groups]
    want, bound, tail, own, all_of_it = reference(
        b,
        lambda s, n: (np.arange(n) >= prefix[s] - 2048) & (np.arange(n) < prefix[s]),  # the prefix's last 2,048 keys
        lambda s, n: (np.arange(n) >= max(prefix[s], n - 1100)) & (np.arange(n) < n - 76),  # a chunk of 1,024 own keys
        lambda s, n: np.arange(n) < prefix[s])
    for wrong, lost in ((np.zeros_like(want), [True] * b.B), (tail, [p >= 2048 for p in prefix]),
                        (own, [n > p + 1200 for n, p in zip(b.n, prefix)]), (all_of_it, [True] * b.B)):
        for s in range(b.B):
            for t in range(int(b.cu[s]), int(b.cu[s + 1])):
                assert not lost[s] or (np.abs(wrong[t] - want[t]) > bound[t]).any(), t
