"""What a chain of ever shorter common prefixes becomes: each link is at least half of its neighbours, and the group's
prefix is the least of all."""
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests import share_ref


def chain(common):
    """Tables of requests that have so many leading blocks in common with the one before, and the step's lengths."""
    width, blocks = max(common) + 1, 0
    tables = []
    for c in [0, *common]:
        row = (tables[-1][:c] if tables else []) + [0] * (width - c)
        for j in range(c, width):
            blocks += 1
            row[j] = blocks
        tables.append(row)
    return list(range(len(tables) + 1)), [4 * width + 1] * len(tables), [t + [-1] for t in tables]


CHAINS = {
    "halves": ([64, 32, 16, 8, 4], [[0, 6, 16]] * 6),  # the prefix is a sixteenth of what the first two share
    "doubles": ([4, 8, 16, 32, 64], [[0, 6, 16]] * 6),
    "less than half": ([64, 31, 16], [[0, 2, 256]] * 2 + [[2, 4, 64]] * 2),
    "half on one side": ([64, 32, 65], [[0, 2, 256]] * 2 + [[2, 4, 260]] * 2),
}


@pytest.mark.parametrize("name", list(CHAINS))
def test_reference(name):
    common, want = CHAINS[name]
    assert share_ref.shared_prefixes(*chain(common), 4, 1) == (want, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CHAINS))
def test_groups(name):
    common, want = CHAINS[name]
    cu, n, tables = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in chain(common))
    assert pkv.pkv_shared_prefixes(cu, n, tables, 4, 1).tolist() == want
    assert pkv.pkv_device_errors() == 0
