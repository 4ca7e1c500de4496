"""The operators around a paged step at the borders of what their calls allow: tensors without elements, streams that are no
torch.cuda.Stream, rows on 16-byte boundaries."""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import paged_step
from test_gpu_paged_step import SITE_RESIZE, Batch, Pool, check_rope, f64, i32, normal, rows_of_many_sizes

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


class Wrapped:
    """A stream as other libraries hand it on: a device and a raw pointer."""

    def __init__(self, stream):
        self.device, self.cuda_stream = stream.device, stream.cuda_stream


def test_streams_of_other_libraries():
    side = torch.cuda.Stream()
    b = Batch([5, 40, 0], 16, 40, 10)
    torch.cuda.synchronize()
    by = [30, -20, 17]
    b.call(by, b.outputs(50), stream=Wrapped(side))
    side.synchronize()
    b.lens, b.table, b.free, *_ = paged_step.resize(by, b.lens, b.table, b.free, 16)
    b.check_state()
    q, pos, rope = normal(1, 20, 3, 64), np.arange(20), mv.Rope(64)
    at, out = i32(pos), torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    for stream in (Wrapped(side), torch.cuda.ExternalStream(side.cuda_stream), side):
        out.fill_(7.0)
        torch.cuda.synchronize()
        mv.qk_norm_rope(q, None, None, None, 1e-6, at, rope, out, stream=stream)
        side.synchronize()
        check_rope(out, q, None, 1e-6, pos, rope)
    far = Wrapped(side)
    for device in (torch.device("cuda", 7), torch.device("cpu"), torch.device("cuda")):
        far.device = device
        with pytest.raises(ValueError, match=f"the stream is on {device},"):
            mv.qk_norm_rope(q, None, None, None, 1e-6, at, rope, out, stream=far)
    for stream in (object(), side.cuda_stream):
        with pytest.raises(AttributeError):
            mv.qk_norm_rope(q, None, None, None, 1e-6, at, rope, out, stream=stream)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("lens,hk", [([1], 1), ([60, 30, 7], 2), ([2000, 1500], 3)])
def test_rows_on_16_byte_boundaries(d, lens, hk):
    """Rows of the caller's that start 16 bytes past a multiple of 32, and whose strides are odd multiples of 16 bytes."""
    pool, t = Pool(lens, hk, d, 16, seed=d), sum(lens)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    # (a buffer starts on a multiple of 32 bytes and more)
    held = [torch.full((t * hk * (d + 8) + 8,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    k, v, ko, vo = (x[8:].view(t, hk, d + 8)[..., :d] for x in held)
    assert all(x.data_ptr() % 32 == 16 and x.stride(1) * 2 % 32 == 16 for x in (k, v, ko, vo))
    k.copy_(rows_of_many_sizes(d, t, hk, d))
    v.copy_(rows_of_many_sizes(d + 1, t, hk, d))
    mv.paged_kv_append(k, v, cu, pool.cache, pool.d_table, pool.d_lens)
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, cu, ko, vo)
    for x, out in ((k, ko), (v, vo)):
        code, byte = paged_step.quantise(f64(x))
        assert np.array_equal(f64(out), paged_step.stored_value(paged_step.pack(code), byte))
    for x in held[2:]:                                         # what lies between stays
        assert (x[:8] == 7.0).all() and (x[8:].view(t, hk, d + 8)[..., d:] == 7.0).all()
