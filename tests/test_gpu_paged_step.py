"""GPU parity of the operators around a paged serving step with the oracle: sequences that grow and shrink, norms of heads
with their rotation, rows held in 4 bits. (Attention over such rows: test_gpu_paged_e2m1.py.)

Tolerances. Whole numbers and what a cache holds are compared exactly. A rotated element may be off its float64 value by
  2^-8 |ref|     its rounding to bf16 (half a step),
  40 2^-24 size  with size the length of its pair: fp32 sums of at most 256 squares in 16 + 4 steps (under a root: 10 units of
                 2^-24), the reciprocal root (2), products with it and the gain (3), the angle (rounded to 2^-24 of at most
                 pi, and its factor: 7), its sine and cosine within 2^-21.1 (7 each), two products and a sum (3), rounded up.
"""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import paged_step

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
SITE_RESIZE = 42


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    mv.lib()


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ growing and shrinking

class Batch:
    """Sequences with their pages, the free stack behind them, and the oracle's copy of both."""

    def __init__(self, lens, page, n_pages, width, seed=0, ld=None):
        r = np.random.default_rng(seed)
        order = r.permutation(n_pages)
        need = [-(-n // page) for n in lens]
        self.page, self.n_pages = page, n_pages
        self.table = r.integers(0, n_pages, (len(lens), width)).astype(np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.lens, self.free = list(lens), [n_pages - at] + order[at:].tolist() + [0] * at
        self.cache = mv.PagedKV.zeros(n_pages, page, 1, 32, mv.DTYPE_E2M1)
        wide = torch.full((len(lens), ld or width), -9, dtype=torch.int32, device="cuda")
        self.d_table = wide[:, :width]
        self.d_table.copy_(i32(self.table))
        self.wide, self.d_lens, self.d_free = wide, i32(lens), i32(self.free)

    def outputs(self, rows):
        n = len(self.lens)
        return (torch.full((n + 1,), 77, dtype=torch.int32, device="cuda"),
                torch.full((rows,), 77, dtype=torch.int32, device="cuda"),
                torch.full((rows,), 77, dtype=torch.int64, device="cuda"))

    def call(self, by, outs=(None, None, None), stream=None):
        mv.paged_kv_resize(i32(by), self.cache, self.d_table, self.d_lens, self.d_free, *outs, stream=stream)

    def check_state(self):
        assert self.d_lens.tolist() == list(self.lens)
        assert self.d_free.tolist() == list(self.free)
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert (self.wide[:, self.table.shape[1]:] == -9).all()

    def step(self, by, extra=3):
        """One call, held against the oracle."""
        rows = sum(max(x, 0) for x in by) + extra
        outs = self.outputs(rows)
        self.call(by, outs)
        self.lens, self.table, self.free, cu, pos, slots = paged_step.resize(by, self.lens, self.table, self.free, self.page)
        self.check_state()
        pad = [-1] * (rows - len(pos))
        assert outs[0].tolist() == cu and outs[1].tolist() == pos + pad and outs[2].tolist() == slots + pad


@pytest.mark.parametrize("n_seq", [1, 2, 31, 33, 511, 512, 513, 1500, 4096])
@pytest.mark.parametrize("page", [16, 48])
def test_resize_random_steps(n_seq, page):
    r = np.random.default_rng(n_seq)
    most = 300 if n_seq < 1000 else 100
    lens = [int(x) for x in r.integers(0, most, n_seq)]
    b = Batch(lens, page, n_seq * 24 + 8, 24, seed=n_seq, ld=29)
    for _ in range(4):
        b.step([int(r.integers(-n, most - n + 1)) if r.random() < 0.6 else 0 for n in b.lens])


@pytest.mark.parametrize("lens,by,page", [
    ([0], [0], 16), ([0], [1], 16), ([16], [1], 16), ([15], [1], 16), ([17], [-1], 16), ([17], [-17], 16),
    ([1024], [0], 1024), ([1, 0, 33], [-1, 48, -33], 16),       # pages given up are taken again in the same call
    ([64, 64], [-64, 64], 16), ([0, 0, 0], [0, 0, 0], 32), ([100], [9000], 16), ([0, 0], [5000, 4001], 128)])
def test_resize_edges(lens, by, page):
    """Lengths at pages' ends, pages that change hands, rows enough for a second kernel."""
    width = max(-(-max(a, a + x) // page) for a, x in zip(lens, by)) or 1
    Batch(lens, page, sum(-(-n // page) for n in lens) + sum(-(-max(0, x) // page) + 1 for x in by), width).step(by)


@pytest.mark.parametrize("rows", [8191, 8192, 8193, 30000])
def test_resize_rows_on_both_sides_of_a_launch(rows):
    b = Batch([5, 0, 77], 16, rows // 16 + 20, rows // 16 + 20, seed=rows)
    b.step([rows - 40, 0, 40], extra=0)
    b.step([-(rows - 41), 3, -100])


def test_resize_back_and_forth_leaves_the_stack():
    r = np.random.default_rng(3)
    b = Batch([int(x) for x in r.integers(0, 500, 40)], 16, 3000, 60)
    before, table = list(b.free), b.d_table.clone()
    by = [int(x) for x in r.integers(0, 300, 40)]
    b.step(by)
    b.step([-x for x in by])
    assert b.free == before
    for s, n in enumerate(b.lens):
        assert torch.equal(b.d_table[s, :-(-n // 16)], table[s, :-(-n // 16)])


@pytest.mark.parametrize("what", ["no_outputs", "cu", "positions", "slots"])
def test_resize_outputs_that_are_not_wanted(what):
    b = Batch([5, 40, 0], 16, 40, 10)
    outs = list(b.outputs(90))
    keep = {"no_outputs": (), "cu": (0,), "positions": (0, 1), "slots": (0, 2)}[what]
    by = [30, -20, 17]
    b.call(by, [o if i in keep else None for i, o in enumerate(outs)])
    b.lens, b.table, b.free, cu, pos, slots = paged_step.resize(by, b.lens, b.table, b.free, 16)
    b.check_state()
    for i, want in enumerate((cu, pos + [-1] * (90 - len(pos)), slots + [-1] * (90 - len(slots)))):
        assert outs[i].tolist() == (want if i in keep else [77] * len(want))


@pytest.mark.parametrize("rows", [200, 9000])
@pytest.mark.parametrize("lens,by,free", [
    ([10, 20], [500, 0], None),                                # more than the table's row holds
    ([10, 20], [-11, 5], None),                                # below nothing
    ([10, -1], [1, 1], None),                                  # a length that is none
    ([10, 20], [2 ** 31 - 1, 5], None), ([10, 20], [-2 ** 31, 5], None),
    ([10, 20], [60, 60], 5),                                   # pages do not suffice
    ([10, 20], [1, 1], -1), ([10, 20], [1, 1], 41),            # a stack of no such size
    ([100, 20], [-60, 0], -1), ([100, 20], [-60, 0], 41), ([100, 20], [0, 0], -2 ** 31), ([100, 20], [0, 0], 2 ** 31 - 1),
    ([100, 20], [-100, 1], 38)])                               # more pages than there are
def test_resize_refused_on_the_device(lens, by, free, rows):
    """Nothing changes, no rows come, the error word says so; the next call is done as ever."""
    b = Batch([max(0, n) for n in lens], 16, 40, 12)
    b.lens = lens
    b.d_lens.copy_(i32(lens))
    if free is not None:
        b.free[0] = free
        b.d_free[0] = free
    outs = b.outputs(rows)
    b.call(by, outs)
    torch.cuda.synchronize()
    st, code = mv.get_error()
    assert st != 0 and code == SITE_RESIZE << 16 | 2
    b.check_state()
    assert outs[0].tolist() == [0] * 3 and (outs[1] == -1).all() and (outs[2] == -1).all()
    b = Batch([10, 20], 16, 40, 12)
    b.step([1, 2])


def test_resize_more_rows_than_there_is_room_for():
    b = Batch([0, 0], 16, 40, 12)
    outs = b.outputs(99)
    b.call([50, 50], outs)
    assert mv.get_error()[0] != 0
    b.check_state()
    assert outs[0].tolist() == [0] * 3 and (outs[1] == -1).all()
    b.step([50, 50], extra=0)


def test_resize_moves_a_bad_page_and_says_so():
    b = Batch([40, 0], 16, 40, 12)
    b.d_table[0, 2] = 1 << 20
    b.table[0, 2] = 1 << 20
    outs = b.outputs(0)
    b.call([-40, 0], outs)
    assert mv.get_error()[0] != 0
    b.lens, b.table, b.free, *_ = paged_step.resize([-40, 0], b.lens, b.table, b.free, 16)
    b.check_state()


def test_resize_of_no_sequences():
    b = Batch([], 16, 4, 3)
    outs = b.outputs(5)
    b.call(np.zeros(0), outs)
    assert outs[0].tolist() == [0] and outs[1].tolist() == [-1] * 5 and outs[2].tolist() == [-1] * 5
    assert b.d_free.tolist() == b.free


def test_resize_replayed_from_a_graph():
    """Both kernels, captured once and replayed as lengths change, on a stream of its own."""
    b = Batch([0, 7, 300], 16, 4000, 1500, seed=5)
    by, rows = i32([0, 0, 0]), 10000
    outs = b.outputs(rows)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mv.paged_kv_resize(by, b.cache, b.d_table, b.d_lens, b.d_free, *outs)
    side = torch.cuda.Stream()
    for step in ([1, 1, 1], [5000, 64, -300], [-4000, 0, 9], [0, -71, 4000]):
        by.copy_(i32(step))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.synchronize()
        b.lens, b.table, b.free, cu, pos, slots = paged_step.resize(step, b.lens, b.table, b.free, 16)
        b.check_state()
        pad = [-1] * (rows - len(pos))
        assert outs[0].tolist() == cu and outs[1].tolist() == pos + pad and outs[2].tolist() == slots + pad


def test_resize_many_calls_in_a_row_and_at_once():
    """Calls that follow each other on a stream without a wait, batches on streams beside each other."""
    r = np.random.default_rng(11)
    jobs = [(Batch([int(x) for x in r.integers(0, 200, n)], 16, n * 60, 50, seed=n), torch.cuda.Stream()) for n in (3, 70, 600)]
    torch.cuda.synchronize()
    steps = [[[int(r.integers(0, 15)) for _ in b.lens] for b, _ in jobs] for _ in range(20)]
    held = [[i32(x) for x in s] for s in steps]
    torch.cuda.synchronize()
    for s, h in zip(steps, held):
        for (b, stream), by, d_by in zip(jobs, s, h):
            mv.paged_kv_resize(d_by, b.cache, b.d_table, b.d_lens, b.d_free, stream=stream)
            b.lens, b.table, b.free, *_ = paged_step.resize(by, b.lens, b.table, b.free, 16)
    torch.cuda.synchronize()
    for b, _ in jobs:
        b.check_state()


# ------------------------------------------------------------------------------------------------ norms and rotation

def freqs_of(rope):
    """Radians for one position, from what the device holds."""
    return [(x % 2 ** 64) / 2.0 ** 64 * 2 * np.pi for x in rope.turns.tolist()] if rope is not None else []


def check_rope(got, x, gain, eps, positions, rope, rows=slice(None)):
    ref, size = paged_step.norm_rope(f64(x), None if gain is None else f64(gain), eps, positions, freqs_of(rope),
                                     rope is not None and rope.neighbours)
    off = np.abs(f64(got) - ref)[rows] / (U * np.abs(ref) + 40 * 2.0 ** -24 * size + 1e-30)[rows]
    assert off.size == 0 or off.max() <= 1.0, f"{off.max():.2f} of the bound"


def run_rope(t, hq, hk, d, rope, seed=0, gain=True, positions=None, eps=1e-6, in_place=False):
    q, k = normal(seed, t, hq, d), normal(seed + 1, t, hk, d, std=3.0)
    qg, kg = (1 + normal(seed + 2, d, std=0.3), normal(seed + 3, d)) if gain else (None, None)
    positions = np.arange(t) if positions is None else positions
    qo, ko = (q.clone(), k.clone()) if in_place else (torch.full_like(q, 7.0), torch.full_like(k, 7.0))
    if in_place:
        mv.qk_norm_rope(qo, ko, qg, kg, eps, i32(positions), rope)
    else:
        mv.qk_norm_rope(q, k, qg, kg, eps, i32(positions), rope, qo, ko)
    torch.cuda.synchronize()
    return q, k, qg, kg, qo, ko, positions


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 256])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("part", ["none", "least", "half", "whole"])
def test_rope_dims(d, neighbours, part):
    rot = {"none": 0, "least": 16, "half": max(16, d // 32 * 16), "whole": d}[part]
    rope = mv.Rope(rot, neighbours=neighbours) if rot else None
    q, k, qg, kg, qo, ko, pos = run_rope(37, 3, 2, d, rope, seed=d)
    check_rope(qo, q, qg, 1e-6, pos, rope)
    check_rope(ko, k, kg, 1e-6, pos, rope)


@pytest.mark.parametrize("t", [1, 2, 3, 33, 456, 457, 1000, 9001])
@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 32), (14, 2), (65, 1), (40, 8)])
def test_rope_tokens_and_heads(t, hq, hk):
    d = 64 if t > 1000 else 128
    rope = mv.Rope(d)
    q, k, qg, kg, qo, ko, pos = run_rope(t, hq, hk, d, rope, seed=t, gain=t % 2 == 0)
    check_rope(qo, q, qg, 1e-6, pos, rope)
    check_rope(ko, k, kg, 1e-6, pos, rope)


def test_rope_many_heads():
    rope = mv.Rope(32)
    q, k, qg, kg, qo, ko, pos = run_rope(5, 256, 256, 32, rope)
    check_rope(qo, q, qg, 1e-6, pos, rope)
    check_rope(ko, k, kg, 1e-6, pos, rope)


@pytest.mark.parametrize("at", [0, 1000, 10 ** 6, 2 ** 31 - 40])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 3.7])
def test_rope_far_positions(at, theta):
    """The oracle's angle in float64 is good to 2^31 2^-53 / 2 radians, far below the bound."""
    rope = mv.Rope(128, theta=theta)
    q, k, qg, kg, qo, ko, pos = run_rope(40, 2, 2, 128, rope, positions=at + np.arange(40), gain=False)
    check_rope(qo, q, qg, 1e-6, pos, rope)
    check_rope(ko, k, kg, 1e-6, pos, rope)


def test_rope_given_frequencies():
    freqs = [0.0, -0.5, 3.0, np.pi, 2 * np.pi + 0.125, 1e-9, 0.1, 100.0]
    rope = mv.Rope(16, freqs=freqs)
    off = np.mod(np.array(freqs_of(rope)) - np.array(freqs) + np.pi, 2 * np.pi) - np.pi
    assert np.abs(off).max() < 1e-13
    q, k, qg, kg, qo, ko, pos = run_rope(300, 2, 1, 32, rope)
    check_rope(qo, q, qg, 1e-6, pos, rope)


@pytest.mark.parametrize("eps", [0.0, 1e-5, 1.0])
def test_rope_eps_and_small_rows(eps):
    rope = mv.Rope(64)
    q, k, qg, kg, qo, ko, pos = run_rope(50, 2, 2, 64, rope, eps=eps)
    check_rope(qo, q, qg, eps, pos, rope)
    z = torch.zeros_like(q)
    out = torch.full_like(q, 7.0)
    mv.qk_norm_rope(z, None, qg, None, max(eps, 1e-6), i32(pos), rope, out)
    assert (out == 0).all()


@pytest.mark.parametrize("by,gain_by,eps", [(57, 100, 1e-6), (57, -100, 0.0), (0, 120, 1e-6), (-55, -100, 0.0), (-55, 100, 0.0)])
@pytest.mark.parametrize("d,rot,neighbours", [(64, 64, False), (128, 64, True), (32, 0, False)])
def test_rope_of_any_size(by, gain_by, eps, d, rot, neighbours):
    """Rows and gains times powers of two, the results within bf16's range: the bound is the one of the gains without theirs.
    (What a product of a gain and a sine loses below 2^-126 is 2^-150, 2^-50 of a row's size.)"""
    rope = mv.Rope(rot, neighbours=neighbours) if rot else None
    pos, gain = np.arange(30), 1 + normal(3, d, std=0.3)
    for h, x in ((3, normal(4, 30, 3, d) * 2.0 ** by), (1, normal(5, 30, 1, d) * 2.0 ** by)):
        out = torch.full_like(x, 7.0)
        mv.qk_norm_rope(x, None, gain * 2.0 ** gain_by, None, eps, i32(pos), rope, out)
        check_rope(out.double() * 2.0 ** -gain_by, x, gain, eps, pos, rope)


@pytest.mark.parametrize("order", ["fused", "planes", "in_place_fused"])
def test_rope_strides(order):
    """Slices of a fused projection, [heads][tokens][D] planes, and a slice in place: what lies between stays."""
    t, hq, hk, d, rope = 70, 6, 2, 96, mv.Rope(64)
    gain = normal(5, d)
    pos = np.arange(t) * 3
    if order == "planes":
        q, k = normal(1, hq, t, d).transpose(0, 1), normal(2, hk, t, d).transpose(0, 1)
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        mv.qk_norm_rope(q, k, gain, gain, 1e-6, i32(pos), rope, qo, ko)
    else:
        x = normal(1, t, hq + 2 * hk, d)
        was = x.clone()
        q, k = was[:, :hq], was[:, hq:hq + hk]
        if order == "fused":
            qo, ko = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hk, d, dtype=torch.bfloat16, device="cuda")
            mv.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], gain, gain, 1e-6, i32(pos), rope, qo, ko)
            assert torch.equal(x, was)
        else:
            qo, ko = x[:, :hq], x[:, hq:hq + hk]
            mv.qk_norm_rope(qo, ko, gain, gain, 1e-6, i32(pos), rope)
            assert torch.equal(x[:, hq + hk:], was[:, hq + hk:])
    check_rope(qo, q, gain, 1e-6, pos, rope)
    check_rope(ko, k, gain, 1e-6, pos, rope)


@pytest.mark.parametrize("rope", [True, False])
def test_rope_leaves_padding(rope):
    r = mv.Rope(128) if rope else None
    pos = np.arange(90)
    pos[[0, 5, 6, 40, 88, 89]] = -1
    real = pos >= 0
    q, k, qg, kg, qo, ko, _ = run_rope(90, 5, 2, 128, r, positions=pos)
    assert (qo[~torch.as_tensor(real)] == 7.0).all() and (ko[~torch.as_tensor(real)] == 7.0).all()
    check_rope(qo, q, qg, 1e-6, pos, r, rows=real)
    check_rope(ko, k, kg, 1e-6, pos, r, rows=real)
    q, k, qg, kg, qo, ko, _ = run_rope(90, 5, 2, 128, r, positions=pos, in_place=True)
    assert torch.equal(qo[~torch.as_tensor(real)], q[~torch.as_tensor(real)])
    check_rope(qo, q, qg, 1e-6, pos, r, rows=real)


def test_rope_rows_stay_to_themselves():
    """A NaN or an infinity reaches its own row alone; one of q or k alone gives the same bits."""
    rope = mv.Rope(64)
    q, k, qg, kg, qo, ko, pos = run_rope(20, 3, 2, 64, rope)
    bad = q.clone()
    bad[7, 1, 5], bad[9, 2, 60] = float("nan"), float("inf")
    out = torch.empty_like(q)
    mv.qk_norm_rope(bad, None, qg, None, 1e-6, i32(pos), rope, out)
    hit = torch.zeros(20, 3, dtype=torch.bool, device="cuda")
    hit[7, 1] = hit[9, 2] = True
    assert torch.equal(out[~hit], qo[~hit]) and torch.isnan(out[7, 1]).all() and torch.isnan(out[9, 2]).any()
    out = torch.empty_like(k)
    mv.qk_norm_rope(None, k, None, kg, 1e-6, i32(pos), rope, None, out)
    assert torch.equal(out, ko)


def test_rope_replayed_and_on_other_streams():
    rope, t = mv.Rope(128), 600
    q, k, qg, kg, qo, ko, pos = run_rope(t, 8, 2, 128, rope)
    d_pos, out, out_k = i32(pos), torch.zeros_like(q), torch.zeros_like(k)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mv.qk_norm_rope(q, k, qg, kg, 1e-6, d_pos, rope, out, out_k)
    for _ in range(2):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, qo) and torch.equal(out_k, ko)
    d_pos += 5
    g.replay()
    torch.cuda.synchronize()
    check_rope(out, q, qg, 1e-6, pos + 5, rope)
    side, outs = torch.cuda.Stream(), [torch.zeros_like(q) for _ in range(6)]
    torch.cuda.synchronize()
    for o in outs:
        mv.qk_norm_rope(q, k, qg, kg, 1e-6, d_pos, rope, o, out_k, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


# ------------------------------------------------------------------------------------------------ rows in 4 bits

class Pool:
    """Sequences over a cache of 4-bit pages in no order."""

    def __init__(self, lens, hk, d, page, seed=0, spare=3):
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + spare
        order, at = r.permutation(n_pages), 0
        self.table = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens, self.hk, self.d, self.page = lens, hk, d, page
        self.cache = mv.PagedKV.zeros(n_pages, page, hk, d, mv.DTYPE_E2M1)
        self.d_table, self.d_lens = i32(self.table), i32(lens)

    def held(self):
        """(packed, bytes) of k and v as the pages hold them."""
        c = self.cache
        return (c.k.cpu().numpy(), c.k_exp.cpu().numpy()), (c.v.cpu().numpy(), c.v_exp.cpu().numpy())

    def place(self, b, p):
        return self.table[b, p // self.page], p % self.page


def rows_of_many_sizes(seed, t, hk, d):
    """Rows whose groups range from nothing to beyond the largest scale, among them exact borders."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((t, hk, d)) * 2.0 ** r.integers(-22, 18, (t, hk, 1)) * 2.0 ** r.integers(-4, 5, (t, hk, d))
    x[r.random((t, hk, d)) < 0.05] = 0.0
    g = x.reshape(t, hk, d // 16, 16)
    half = r.random((t, hk, d // 16)) < 0.3                    # groups of values on borders of some scale
    s = paged_step.scale_value(r.integers(1, paged_step.TOP_BYTE + 1, (t, hk, d // 16)))[..., None]
    b = np.array([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -0.75, -2.5])
    g = np.where(half[..., None], b * s, g)
    return torch.tensor(g.reshape(t, hk, d)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("lens,counts,hk,page", [
    ([1], [1], 1, 16), ([40, 7, 0, 129], [40, 7, 0, 129], 3, 16), ([500, 33], [20, 1], 2, 48), ([2000, 1500, 7], [2000, 1500, 7], 8, 64),
    ([1025] * 5, [1] * 5, 4, 1024)])
def test_rows_written_and_read(d, lens, counts, hk, page):
    pool = Pool(lens, hk, d, page, seed=d)
    cu = np.concatenate([[0], np.cumsum(counts)])
    t = int(cu[-1])
    k, v = rows_of_many_sizes(d, t, hk, d), rows_of_many_sizes(d + 1, t, hk, d)
    mv.paged_kv_append(k, v, i32(cu), pool.cache, pool.d_table, pool.d_lens)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32(cu), ko, vo)
    torch.cuda.synchronize()
    for x, out, (pages, bytes_) in zip((k, v), (ko, vo), pool.held()):
        code, byte = paged_step.quantise(f64(x))
        packed, seen = paged_step.pack(code), np.zeros(bytes_.shape[:3], dtype=bool)
        assert np.array_equal(f64(out), paged_step.stored_value(packed, byte))
        for b, (n, c) in enumerate(zip(lens, counts)):
            for i in range(c):
                at, slot = pool.place(b, n - c + i)
                seen[at, :, slot] = True
                value = paged_step.stored_value(pages[at, :, slot], bytes_[at, :, slot])
                assert np.array_equal(bytes_[at, :, slot], byte[cu[b] + i])
                assert np.array_equal(value, paged_step.stored_value(packed[cu[b] + i], byte[cu[b] + i]))
        assert not pages[~seen].any() and not bytes_[~seen].any()   # nothing else is written


def test_rows_with_nan_and_infinity():
    pool = Pool([20], 2, 64, 16)
    k = normal(1, 20, 2, 64)
    k[3, 0, 5], k[4, 1, 63], k[5, 0, 0], k[5, 0, 1] = float("nan"), float("inf"), float("-inf"), float("nan")
    k[6, 1] = 3.3e38
    mv.paged_kv_append(k, k, i32([0, 20]), pool.cache, pool.d_table, pool.d_lens)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32([0, 20]), ko, vo)
    code, byte = paged_step.quantise(f64(k))
    want = paged_step.stored_value(paged_step.pack(code), byte)
    assert np.array_equal(f64(ko), want, equal_nan=True) and np.array_equal(f64(vo), want, equal_nan=True)
    assert np.isnan(want).sum() == 48 and (want[6, 1] == 61440).all()


def test_rows_every_byte_read_back():
    """All scale bytes, also those that are never written, with all 16 codes."""
    pool = Pool([256], 1, 32, 256)
    pool.cache.k.copy_((torch.arange(16, dtype=torch.uint8, device="cuda") * 17).expand(pool.cache.k.shape))
    at = pool.place(0, 0)[0]
    pool.cache.k_exp[at, 0] = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None]
    ko, vo = (torch.empty(256, 1, 32, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32([0, 256]), ko, vo)
    byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None, None], 2, axis=2)
    with np.errstate(invalid="ignore"):
        want = paged_step.stored_value(np.broadcast_to((np.arange(16) * 17).astype(np.uint8), (256, 1, 16)), byte)
    assert np.array_equal(f64(ko), want, equal_nan=True)


def test_rows_of_other_strides():
    pool = Pool([60, 30], 2, 96, 16)
    x = rows_of_many_sizes(4, 90, 8, 96)
    k, v = x[:, 2:4], x[:, 6:8]
    mv.paged_kv_append(k, v, i32([0, 60, 90]), pool.cache, pool.d_table, pool.d_lens)
    planes = torch.full((2, 2, 90, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32([0, 60, 90]), planes[0].transpose(0, 1), planes[1].transpose(0, 1))
    for x, out in ((k, planes[0]), (v, planes[1])):
        code, byte = paged_step.quantise(f64(x))
        assert np.array_equal(f64(out.transpose(0, 1)), paged_step.stored_value(paged_step.pack(code), byte))


def test_rows_of_a_bad_page_are_left_out():
    pool = Pool([40, 20], 2, 64, 16)
    table = pool.d_table.clone()
    table[0, 1] = pool.cache.n_pages
    k = normal(3, 60, 2, 64)
    mv.paged_kv_append(k, k, i32([0, 40, 60]), pool.cache, table, pool.d_lens)
    assert mv.get_error()[0] != 0
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    mv.paged_kv_read(pool.cache, table, pool.d_lens, i32([0, 40, 60]), ko, vo)
    assert mv.get_error()[0] != 0
    code, byte = paged_step.quantise(f64(k))
    want = paged_step.stored_value(paged_step.pack(code), byte)
    want[16:32] = 7.0
    assert np.array_equal(f64(ko), want)


# ------------------------------------------------------------------------------------------------ what the binding refuses

def test_refusals_with_tensors():
    """Wrong types, sizes, layouts and tensors of the host: an error before anything is launched, and nothing is written."""
    b = Batch([5, 40], 16, 40, 10)
    by, (cu, pos, slots) = i32([1, 1]), b.outputs(8)
    call = lambda by=by, table=b.d_table, lens=b.d_lens, free=b.d_free, cu=cu, pos=pos, slots=slots, **kw: \
        mv.paged_kv_resize(by, b.cache, table, lens, free, cu, pos, slots, **kw)
    for kw in (dict(by=by.long()), dict(by=i32([1, 1, 1])), dict(by=by.cpu()), dict(table=b.d_table.long()), dict(table=b.d_table[0]),
               dict(table=b.d_table.t()), dict(lens=b.d_lens[:1]), dict(free=b.d_free[:-1]), dict(cu=cu[:2]), dict(cu=None), dict(pos=pos[::2]),
               dict(pos=pos.long()), dict(slots=slots.int()), dict(slots=slots[:7]), dict(slots=slots[None]), dict(by=[1, 1])):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    b.check_state()
    assert (cu == 77).all() and (pos == 77).all() and (slots == 77).all()

    q, k, gain, at, rope = normal(1, 4, 3, 64), normal(2, 4, 2, 64), normal(3, 64), i32(range(4)), mv.Rope(64)
    out = torch.full_like(q, 7.0)
    turn = lambda q=q, k=k, qg=gain, kg=gain, at=at, rope=rope, qo=out, ko=None, eps=1e-6: \
        mv.qk_norm_rope(q, k, qg, kg, eps, at, rope, qo, ko)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q.cpu()), dict(k=normal(2, 5, 2, 64)), dict(k=normal(2, 4, 2, 32)),
               dict(q=normal(1, 4, 3, 128)[..., ::2]), dict(qg=gain.float()), dict(kg=gain[:32]), dict(at=at.long()), dict(at=at[:3]), dict(at=None),
               dict(qo=out[:, :2]), dict(q=None), dict(rope=mv.Rope(64, device="cpu"))):
        with pytest.raises((ValueError, TypeError)):
            turn(**kw)
    for kw in (dict(rope=mv.Rope(128)), dict(eps=-1.0), dict(q=normal(1, 4, 3, 72)[..., 4:68].contiguous()[:, :, :56], k=None, kg=None, qg=None)):
        with pytest.raises((ValueError, mv.MVError)):
            turn(**kw)
    assert (out == 7.0).all()

    pages = torch.zeros(4, 2, 16, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(4, 2, 16, 4, dtype=torch.uint8, device="cuda")
    mv.PagedKV(pages, pages.clone(), scales, scales.clone())
    for args in ((pages, pages, None, None), (pages, pages, scales, None), (pages, pages, scales[..., :3], scales[..., :3]),
                 (pages, pages, scales[..., 0].contiguous(), scales[..., 0].contiguous()), (pages, pages.to(torch.int8), scales, scales),
                 (pages.transpose(1, 2), pages.transpose(1, 2), scales, scales), (pages, pages, scales.int(), scales.int())):
        with pytest.raises(ValueError):
            mv.PagedKV(*args)
