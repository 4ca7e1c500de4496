"""The operators around a paged step at the borders of what their calls allow: tensors without elements."""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import paged_step
from test_gpu_paged_step import SITE_RESIZE, Batch, i32, normal

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


@pytest.mark.parametrize("rope", [True, False])
def test_heads_of_no_tokens(rope):
    """A step without rows: nothing to do, whether or not the heads would be turned."""
    q, k = normal(1, 0, 4, 64), normal(2, 0, 2, 64)
    gain, at, r = normal(3, 64), i32([]), mv.Rope(64) if rope else None
    mv.qk_norm_rope(q, k, gain, gain, 1e-6, at, r)
    mv.qk_norm_rope(q, None, gain, None, 1e-6, at, r, torch.empty_like(q))
    with pytest.raises(ValueError):
        mv.qk_norm_rope(q, k, gain, gain, 1e-6, None, mv.Rope(64))   # a rotation wants positions, be it of no tokens
    q = normal(1, 3, 4, 64)
    out = torch.full_like(q, 7.0)
    with pytest.raises(ValueError):
        mv.qk_norm_rope(q, None, gain, None, 1e-6, at, r, out)       # no positions for three tokens
    assert (out == 7.0).all()
