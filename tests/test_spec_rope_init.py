"""Settings of a rotary embedding whose angles leave the numbers are refused,
those at the edge keep the formula (host only)."""
import math

import pytest

import paged_kv_cache_mapping_gb300 as pkv
from paged_kv_cache_mapping_gb300 import build as pkv_build

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv_build.build()


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=5e-324), dict(scaling="linear", factor=1e-309),  # 1 / factor overflows
    dict(scaling="smooth", factor=1e-309, original_max_position=10),
    dict(scaling="by_parts", factor=1e-309, original_max_position=10),
    dict(rot_dim=4, scaling="ntk", factor=1e200),   # base * factor^2
    dict(rot_dim=4, scaling="ntk", factor=1e-200),
    dict(rot_dim=256, base=1.0000001, scaling="ntk", factor=5e-324),
    dict(attention_factor=1e39), dict(attention_factor=NAN),
    dict(scaling="by_parts", factor=2.0, original_max_position=100, fast=NAN),
    dict(scaling="by_parts", factor=2.0, original_max_position=100, slow=-1.0),
    dict(scaling="smooth", factor=2.0, original_max_position=100, fast=-4.0),
    dict(scaling="smooth", factor=2.0, original_max_position=INF),
])
def test_refused(kw):
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_rope_init(**{"rot_dim": 64, **kw})
    assert e.value.status == 1


def test_edges():
    tiny = pkv.pkv_rope_init(64, scaling="linear", factor=1e-300)  # 1e300 radians a position, modulo one turn
    want = (1e300 / (2 * math.pi)) % 1.0
    assert tiny.turns[0] / 2.0 ** 64 == want
    assert pkv.pkv_rope_init(64, attention_factor=3e38).amplitude > 2.9e38
    # a factor of one or less stretches nothing: no correction of the amplitude
    assert pkv.pkv_rope_init(64, scaling="by_parts", factor=0.5, original_max_position=4096).amplitude == 1.0
    assert pkv.pkv_rope_init(64, scaling="by_parts", factor=1.0, original_max_position=4096).amplitude == 1.0
    two = pkv.pkv_rope_init(2, scaling="ntk", factor=8.0)  # one pair: its angle is the position for any base
    assert abs(two.turns[0] / 2.0 ** 64 - 1 / (2 * math.pi)) < 2.0 ** -52
