"""The operators around a paged step at the borders of what their calls allow: tensors without elements."""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import paged_step
from test_gpu_paged_step import SITE_RESIZE, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    mv.lib()


@pytest.mark.parametrize("what", ["positions", "slots", "both"])
@pytest.mark.parametrize("room", [0, 1])
def test_resize_into_room_for_fewer_rows(what, room):
    """Positions or slots with room for no row, or for one, are as much of a limit as any: nothing is done, and a call that
    lets nothing come is."""
    b = Batch([5, 40], 16, 40, 10)
    cu, pos, slots = b.outputs(room)
    outs = (cu, None if what == "slots" else pos, None if what == "positions" else slots)
    b.call([1, 1], outs)
    torch.cuda.synchronize()
    st, code = mv.get_error()
    assert st != 0 and code == SITE_RESIZE << 16 | 2
    b.check_state()
    assert cu.tolist() == [0] * 3
    b.call([0, -20], outs)
    assert mv.get_error()[0] == 0
    b.lens, b.table, b.free, *_ = paged_step.resize([0, -20], b.lens, b.table, b.free, 16)
    b.check_state()
    for x, given in ((pos, what != "slots"), (slots, what != "positions")):
        assert x.tolist() == [-1 if given else 77] * room
