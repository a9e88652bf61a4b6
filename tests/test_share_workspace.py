"""What the workspace of shared attention grows with (no GPU)."""
import pytest

from tests.test_abi import BF16, E4M3, I32
from tests.test_share_refusals import at, attention_args, lib, workspace  # noqa: F401  (lib: a fixture)


def size(lib, B, T, blocks, max_q=0, max_group=0, Hq=32, Hkv=8, D=128, cdt=BF16):  # noqa: F811
    a = attention_args(T=T, Hq=Hq, Hkv=Hkv, D=D, B=B, cdt=cdt)
    return workspace(lib, {**a, "bt": at(4, I32, [B, blocks]), "max_q": max_q, "max_g": max_group})


@pytest.mark.parametrize("cdt", [BF16, E4M3])
@pytest.mark.parametrize("B,T,max_q,max_group,chunks", [
    (256, 256, 0, 0, 8),           # decodes, bounds unknown
    (257, 2256, 2000, 2256, 8),    # one prompt among decodes
    (8192, 8192, 0, 0, 8),         # as many as a step has
    (64, 64, 0, 0, 8),
])
def test_it_holds_no_more_rows_than_the_batch_can_fill(lib, cdt, B, T, max_q, max_group, chunks):  # noqa: F811
    """Each row has at most `chunks` partials of its own keys (this many heads cut no finer), at most 4,096 partials of
    prefixes are left in all, and one more."""
    row = 4 * 32 * 129
    n = size(lib, B, T, 8192, max_q, max_group, cdt=cdt)  # 131,072 tokens a table
    assert n <= (T * chunks + max(4096, T) + T) * row + 32 * B + 512


def test_it_counts_requests_where_most_rows_are_padding(lib):  # noqa: F811
    row = 4 * 32 * 129
    assert size(lib, 64, 1 << 20, 8192, 1, 64) <= (64 * 8 + 2 * (1 << 20)) * row + 32 * 64 + 512
