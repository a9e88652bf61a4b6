"""Long steps (four rows a thread) whose slots and positions do not lie on 16
bytes, or that ask for no positions."""
import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from tests.test_gpu_step_tables import DEV, step

pytestmark = pytest.mark.gpu


def place(x, off):
    """x as a view `off` elements into a buffer, and the buffer."""
    buf = torch.full((x.shape[0] + 8,), -55, dtype=x.dtype, device=DEV)
    buf[off:off + x.shape[0]] = x
    return buf[off:off + x.shape[0]], buf


@pytest.mark.parametrize("i64", [False, True])
@pytest.mark.parametrize("slots,positions", [(1, 0), (0, 1), (2, 2), (3, 1), (4, 4), (0, None), (1, None)])
@pytest.mark.parametrize("B,grow,pad", [(40, 90, 5), (9, 2000, 0), (3, 9000, 1), (300, 40, 3)])
def test_placement(B, grow, pad, slots, positions, i64):
    st = step(1000 + B, B, 16, 300, grow, T_pad=pad, shared=True, i64=i64, positions=positions is not None)
    T = st.slots.shape[0]
    assert T > 1024
    st.slots, slot_buf = place(st.slots, slots)
    st.args = (*st.args[:7], st.slots)
    pos_buf = None
    if positions is not None:
        st.pos, pos_buf = place(st.pos, positions)
        st.kw["positions"] = st.pos
    st.run()
    st.check()
    for buf, off in ((slot_buf, slots), (pos_buf, positions)):
        if buf is not None:
            assert (buf[:off] == -55).all() and (buf[off + T:] == -55).all()


def test_the_long_prompt_alone_without_positions():
    st = step(7, 2, 12, 30, 5000, i64=False, positions=False)
    assert st.slots.shape[0] > 1024
    st.run()
    st.check()
    assert pkv.pkv_device_errors() == 0
