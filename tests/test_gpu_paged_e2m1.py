"""GPU parity of one-token attention over a cache of 4-bit rows with the oracle, and of a serving step's operators one after
the other.

Tolerances. What pages stand for is exact, so an element may be off its float64 value by
  2^-8 |ref|                        the result's rounding to bf16 (half a step),
  (2^-11 + 2 s + (n + 8) 2^-23) A   with A = sum_j p_j |v_j|: the weights' rounding to fp16 (half a step; weights below its
                                    normal range go as two bf16, 2^-16), the error s of an exponent, (D + 8) 2^-23 scale
                                    max_j sum_d |q_d k_jd| for products summed in fp32 plus the rounding of the exponent
                                    itself, and fp32 sums over n keys.
"""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import paged_step, serving
from test_gpu_paged_step import Pool, f64, i32, normal

pytestmark = pytest.mark.gpu
U, W = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    mv.lib()


def fill(pool, seed, k_std=1.0, k=None, v=None):
    """Whole sequences of rows written."""
    t = sum(pool.lens)
    k = normal(seed, t, pool.hk, pool.d, std=k_std) if k is None else k
    v = normal(seed + 1, t, pool.hk, pool.d) if v is None else v
    cu = np.concatenate([[0], np.cumsum(pool.lens)])
    mv.paged_kv_append(k, v, i32(cu), pool.cache, pool.d_table, pool.d_lens)
    return pool


def run(pool, q, scale, out=None, ws=None, stream=None):
    out = torch.full_like(q, 7.0) if out is None else out
    if ws is None:
        ws = torch.zeros(mv.paged_attention_workspace(len(q), q.shape[1], pool.hk, pool.d), dtype=torch.uint8, device="cuda")
    mv.paged_attention(q, pool.cache, pool.d_table, pool.d_lens, scale, out, ws, stream=stream)
    return out


def sequence(pool, b, held):
    """Rows [len, Hk, D] of what sequence b's pages stand for."""
    n, (packed, byte) = pool.lens[b], held
    ids = pool.table[b, :-(-n // pool.page)]
    x = paged_step.stored_value(packed[ids], byte[ids])
    return x.transpose(0, 2, 1, 3).reshape(len(ids) * pool.page, pool.hk, pool.d)[:n]


def check(pool, q, out, scale):
    held = pool.held()
    q, out = f64(q), f64(out)
    group = q.shape[1] // pool.hk
    for b, n in enumerate(pool.lens):
        k, v = sequence(pool, b, held[0]), sequence(pool, b, held[1])
        for c in range(pool.hk):
            rows = slice(c * group, (c + 1) * group)
            ref, mag = serving.attend(q[b, rows], k[:, c], v[:, c], scale, np.ones((group, n), dtype=bool))
            dots = scale * np.max(np.abs(q[b, rows]) @ np.abs(np.where(np.isfinite(k[:, c]), k[:, c], 0)).T, axis=1, initial=0.0)
            s = ((pool.d + 8) * 2.0 ** -23 * dots)[:, None]
            tol = U * np.abs(ref) + (W + 2 * s + (n + 8) * 2.0 ** -23) * mag + 1e-30
            fin = np.isfinite(ref)
            assert np.array_equal(fin, np.isfinite(out[b, rows]))
            off = (np.abs(out[b, rows] - ref)[fin] / tol[fin]).max(initial=0.0)
            assert off <= 1.0, f"sequence {b}, kv head {c}: {off:.2f} of the bound"


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [513], [1027], [4000], [0], [0, 3, 0],
                                  [1, 600, 0, 33, 2100], [64, 64, 64], [1500] * 5])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 128), (8, 2, 128), (5, 1, 64)])
def test_lengths(lens, hq, hk, d):
    pool = fill(Pool(lens, hk, d, 16, seed=len(lens)), 1)
    q = normal(3, len(lens), hq, d)
    check(pool, q, run(pool, q, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 1), (9, 1), (16, 2), (17, 1), (40, 2), (32, 32), (14, 2)])
def test_groups_and_dims(hq, hk, d):
    lens = [700, 9, 130]
    pool = fill(Pool(lens, hk, d, 32, seed=d), d)
    q = normal(7, 3, hq, d)
    check(pool, q, run(pool, q, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 112, 128, 1024])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(page, d):
    lens = [1300, 47, 2 * page + 1]
    pool = fill(Pool(lens, 2, d, page, seed=page), page)
    q = normal(5, 3, 4, d)
    check(pool, q, run(pool, q, 0.2), 0.2)


@pytest.mark.parametrize("n_seq,hq,hk,d,most", [(1, 16, 2, 128, 40000), (1, 32, 32, 128, 1027), (1, 8, 8, 64, 9000), (12, 16, 1, 128, 5000),
                                                (70, 8, 4, 64, 900), (200, 8, 8, 128, 300), (1100, 2, 2, 64, 60)])
def test_many_steps_and_sequences(n_seq, hq, hk, d, most):
    """Units that cross CTAs, clusters for one sequence, a unit to each warp, more sequences than a launch takes."""
    r = np.random.default_rng(n_seq)
    lens = [most] + [int(x) for x in r.integers(0, most + 1, n_seq - 1)]
    pool = fill(Pool(lens, hk, d, 64, seed=n_seq), n_seq)
    q = normal(5, n_seq, hq, d)
    out = run(pool, q, d ** -0.5)
    check(pool, q, out, d ** -0.5)
    for _ in range(3):
        assert torch.equal(run(pool, q, d ** -0.5), out)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (0.5, 3.0), (1.0, 6.0), (1e-3, 1.0), (1.0, 60.0)])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 128), (20, 2, 64)])
def test_scales(scale, std, hq, hk, d):
    """Uniform weights, and scores far enough apart that weights leave fp16's range."""
    pool = fill(Pool([900, 5, 300], hk, d, 16), 9, k_std=std)
    q = normal(2, 3, hq, d, std=std)
    check(pool, q, run(pool, q, scale), scale)


@pytest.mark.parametrize("drop", [5.0, 12.0, 20.0, 28.0, 45.0, 80.0])
@pytest.mark.parametrize("where", [0, 100, 511, 1999])
def test_columns_of_small_weights_alone(drop, where):
    """Each column of V has something in one key only; the weights fall by 2^-drop from the first keys to that one."""
    n, d, hk = 2000, 64, 1
    k = torch.zeros(n, hk, d, device="cuda")
    k[:, :, 0] = 6.0
    k[where, :, 0] = -6.0
    v = torch.zeros(n, hk, d, device="cuda")
    v[(where + 1) % n, 0, :32] = 3.0
    v[where, 0, 32:] = 2.0
    pool = fill(Pool([n], hk, d, 16), 0, k=k.to(torch.bfloat16), v=v.to(torch.bfloat16))
    q = torch.zeros(1, 2, d, device="cuda")
    q[:, :, 0] = 1.0
    q[:, 1, 0] = 0.5
    q = q.to(torch.bfloat16)
    scale = drop * np.log(2) / 12
    out = run(pool, q, scale)
    assert (out[0, :, 32:] > 0).all()
    check(pool, q, out, float(np.float32(scale)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,k0", [(1.0, 4096.0), (0.125, 4.0), (1.0, -4096.0), (2.0 ** 30, 4096.0), (1e30, 2.0 ** -10), (0.0, 64.0),
                                      (1e-37, 64.0), (2.0 ** -9, 4.0)])
@pytest.mark.parametrize("lens", [[400], [5000, 33]])
def test_scores_of_any_size(d, scale, k0, lens):
    """Scores that fp32 holds exactly: each is one product, about 2^20 k0 times 1, 1.5 or 2, times the scale. So weights are
    known to the rounding of an exponent of at most 2^-23 |score|, and where the scores differ by more than 2^9 they are 0
    and 1."""
    t, hq, hk = sum(lens), 2, 1
    k = torch.zeros(t, hk, d, device="cuda")
    k[:, :, 0] = k0 * (1 + (torch.arange(t, device="cuda") * 5 % 3)[:, None] / 2)
    pool = fill(Pool(lens, hk, d, 16), 2, k=k.to(torch.bfloat16))
    held = pool.held()[0]
    q = torch.zeros(len(lens), hq, d, device="cuda")
    q[:, :, 0] = 2.0 ** 20
    q = q.to(torch.bfloat16)
    out = f64(run(pool, q, scale))
    scale = float(np.float32(scale))
    top = abs(k0) * 2.0 ** 21.1 * scale                       # more than the largest score's size
    assert top < 2.0 ** 14 or top / 8 > 2.0 ** 9
    for b, n in enumerate(lens):
        kk, vv = sequence(pool, b, held)[:, 0], sequence(pool, b, pool.held()[1])[:, 0]
        sizes = np.unique(np.abs(kk[:, 0])) / abs(k0)         # what 4 bits make of 1, 1.5 and 2: an eighth of top apart or more
        assert len(sizes) <= 3 and sizes[-1] < 2.1 and (np.diff(sizes) > 0.4).all()
        ref, mag = serving.attend(f64(q[b]), kk, vv, scale, np.ones((hq, n), dtype=bool))
        tol = U * np.abs(ref) + (W + (top * 2.0 ** -21 if top < 2.0 ** 14 else 0.0) + (n + 8) * 2.0 ** -23) * mag
        assert (np.abs(out[b] - ref) <= tol).all()


def test_rising_scores():
    """Each later key scores higher, so every step moves the reference."""
    n, d = 3000, 64
    k = (torch.arange(n, device="cuda")[:, None, None] * 0.02).expand(n, 1, d).to(torch.bfloat16).contiguous()
    pool = fill(Pool([n], 1, d, 16), 3, k=k)
    q = torch.ones(1, 2, d, dtype=torch.bfloat16, device="cuda")
    check(pool, q, run(pool, q, 0.3), 0.3)


@pytest.mark.parametrize("d", [96, 128])
def test_scales_of_any_byte(d):
    """Groups whose scales lie 2^27 apart, subnormal ones among them, in K and in V."""
    r = np.random.default_rng(d)
    pool = Pool([300, 20], 2, d, 16)
    c = pool.cache
    for x in (c.k, c.v):
        x.copy_(torch.as_tensor(r.integers(0, 256, tuple(x.shape)), dtype=torch.uint8))
    c.k_exp.copy_(torch.as_tensor(r.integers(0, 130, tuple(c.k_exp.shape)), dtype=torch.uint8))
    c.v_exp.copy_(torch.as_tensor(r.integers(0, 0xE3, tuple(c.v_exp.shape)), dtype=torch.uint8))
    q = normal(1, 2, 4, d)
    check(pool, q, run(pool, q, 0.05), 0.05)


def test_queries_of_any_size():
    pool = fill(Pool([200], 1, 64, 16), 4)
    for std in (1e-30, 1e-5, 1e5, 1e30):
        q = normal(8, 1, 3, 64, std=std)
        check(pool, q, run(pool, q, 1.0 / std), float(np.float32(1.0 / std)))


@pytest.mark.parametrize("d", [96, 128])
@pytest.mark.parametrize("lens", [[1], [20], [130, 64, 15], [1000]])
def test_what_lies_behind_a_sequence_does_not_matter(d, lens):
    """Scale bytes 255 and codes of anything behind the length, in the rest of its page and in every other page."""
    pool = fill(Pool(lens, 2, d, 64, seed=2), 6)
    q = normal(3, len(lens), 8, d)
    want = run(pool, q, 0.1)
    check(pool, q, want, 0.1)
    c = pool.cache
    mine = torch.zeros(c.n_pages, 64, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for p in range(n):
            at, slot = pool.place(b, p)
            mine[at, slot] = True
    for x, value in ((c.k, 0x77), (c.v, 0x77), (c.k_exp, 255), (c.v_exp, 255)):
        x.permute(0, 2, 1, 3)[~mine] = value
    assert torch.equal(run(pool, q, 0.1), want)


def test_nan_groups_reach_their_own():
    """A NaN in a value group reaches that group's columns of its head's rows; in a key, all of the head's rows."""
    pool = fill(Pool([90, 40], 2, 128, 16), 6)
    q = normal(3, 2, 4, 128)
    want = run(pool, q, 0.1)
    at, slot = pool.place(0, 50)
    pool.cache.v_exp[at, 1, slot, 3] = 255
    out = run(pool, q, 0.1)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 2:, 48:64] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], want[~hit])
    at, slot = pool.place(1, 7)
    pool.cache.k_exp[at, 0, slot, 0] = 255
    out = run(pool, q, 0.1)
    hit[1, :2] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("lens", [[300, 40, 70], [5000, 64, 3000]])
def test_bad_pages_and_lengths_keep_their_rows(lens):
    pool = fill(Pool(lens, 2, 64, 16), 6)
    q = normal(3, 3, 4, 64)
    want = run(pool, q, 0.1)
    good = pool.d_table.clone()
    for bad in (-1, pool.cache.n_pages, 2 ** 31 - 1):
        pool.d_table[0, 2] = bad
        out = run(pool, q, 0.1)
        assert mv.get_error()[0] != 0
        assert (out[0] == 7.0).all() and torch.equal(out[1:], want[1:])
    pool.d_table.copy_(good)
    for bad in (-1, pool.d_table.shape[1] * 16 + 1):
        pool.d_lens[1] = bad
        out = run(pool, q, 0.1)
        assert mv.get_error()[0] != 0
        assert (out[1] == 7.0).all() and torch.equal(out[::2], want[::2])
    pool.d_lens[1] = lens[1]
    assert torch.equal(run(pool, q, 0.1), want)


def test_strides_of_q_and_out():
    pool = fill(Pool([100, 40], 2, 96, 16), 6)
    x = normal(3, 2, 12, 96)
    wide = torch.full((2, 9, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    run(pool, x[:, 3:7], 0.1, out=wide[:, 1:5])
    check(pool, x[:, 3:7], wide[:, 1:5], 0.1)
    assert (wide[:, 0] == 7.0).all() and (wide[:, 5:] == 7.0).all()


def test_calls_at_once_and_replayed():
    """Streams beside each other, each with a workspace of its own, and graphs between them as lengths change."""
    jobs = []
    for seed, (lens, hq, hk, d) in enumerate([([3000, 5], 8, 2, 128), ([2000], 32, 32, 64), ([900] * 7 + [0], 6, 2, 128)]):
        pool = fill(Pool(lens, hk, d, 16, seed=seed), seed)
        q = normal(3, len(lens), hq, d)
        ws = torch.zeros(mv.paged_attention_workspace(len(lens), hq, hk, d), dtype=torch.uint8, device="cuda")
        want = run(pool, q, 0.1, ws=ws)
        jobs.append((pool, q, ws, want, [torch.full_like(want, float("nan")) for _ in range(6)], torch.cuda.Stream()))
    pool, q, *_ = jobs[0]
    ws, graphed = torch.zeros_like(jobs[0][2]), torch.zeros_like(jobs[0][3])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run(pool, q, 0.1, out=graphed, ws=ws)
    for i in range(6):
        for p, x, w, _, outs, stream in jobs:
            run(p, x, 0.1, out=outs[i], ws=w, stream=stream)
        g.replay()
    torch.cuda.synchronize()
    for _, _, _, want, outs, _ in jobs:
        assert all(torch.equal(o, want) for o in outs)
    assert torch.equal(graphed, jobs[0][3])
    pool.lens = [1700, 3]
    pool.d_lens.copy_(i32(pool.lens))
    g.replay()
    torch.cuda.synchronize()
    check(pool, q, graphed, 0.1)


def test_pool_of_more_than_32_bits_of_bytes():
    """Rows whose offset in the pool passes 2^32 bytes, and whose scales pass 2^31."""
    hk, d, page = 64, 128, 1024
    n_pages = 2 ** 32 // (hk * page * d // 2) + 3
    cache = mv.PagedKV.zeros(n_pages, page, hk, d, mv.DTYPE_E2M1)
    table = i32([[n_pages - 1, n_pages - 2]])
    lens, rows = i32([1100]), normal(1, 1100, hk, d)
    mv.paged_kv_append(rows, rows, i32([0, 1100]), cache, table, lens)
    back = torch.empty_like(rows)
    mv.paged_kv_read(cache, table, lens, i32([0, 1100]), back, torch.empty_like(rows))
    assert cache.k[:-2].max() == 0 and cache.k_exp[:-2].max() == 0
    q, out = normal(2, 1, hk, d), torch.empty(1, hk, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mv.paged_attention_workspace(1, hk, hk, d), dtype=torch.uint8, device="cuda")
    mv.paged_attention(q, cache, table, lens, 0.1, out, ws)
    for h in (0, 33, 63):
        x = f64(back[:, h])
        assert np.array_equal(x, paged_step.stored_value(*[f(y) for f, y in zip((paged_step.pack, lambda b: b), paged_step.quantise(f64(rows[:, h])))]))
        ref, mag = serving.attend(f64(q[0, h:h + 1]), x, x, 0.1, np.ones((1, 1100), dtype=bool))
        tol = U * np.abs(ref) + (W + 2 * 136 * 2.0 ** -23 * 0.1 * 128 * 16 + 1108 * 2.0 ** -23) * mag
        assert (np.abs(f64(out[0, h:h + 1]) - ref) <= tol).all()


# ------------------------------------------------------------------------------------------------ a serving step

@pytest.mark.parametrize("dtype", [mv.DTYPE_BF16, mv.DTYPE_E4M3, mv.DTYPE_E2M1])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(dtype, graph):
    """Requests that take and give up tokens: tables, rotated heads, cache rows and attention over them, step after step; from
    a graph with a fixed number of rows, padded. Every step against the oracle's own tables and rows."""
    page, n_pages, hq, hk, d, n_seq, n_rows = 16, 80, 6, 2, 64, 4, 48
    cache = mv.PagedKV.zeros(n_pages, page, hk, d, dtype)
    table, lens = i32(np.zeros((n_seq, 16))), i32(np.zeros(n_seq))
    free = i32([n_pages] + list(range(n_pages)))
    by, rope, gain = i32(np.zeros(n_seq)), mv.Rope(d), 1 + normal(1, d, std=0.2)
    cu, positions = i32(np.zeros(n_seq + 1)), i32(np.zeros(n_rows))
    slots = torch.zeros(n_rows, dtype=torch.int64, device="cuda")
    qkv = torch.zeros(n_rows, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    last, out = torch.zeros(n_seq, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n_seq, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mv.paged_attention_workspace(n_seq, hq, hk, d), dtype=torch.uint8, device="cuda")
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]

    def step():
        mv.paged_kv_resize(by, cache, table, lens, free, cu, positions, slots)
        mv.qk_norm_rope(q, k, gain, gain, 1e-6, positions, rope)
        mv.paged_kv_append(k, v, cu, cache, table, lens)
        mv.paged_attention(last, cache, table, lens, 0.125, out, ws)

    g = torch.cuda.CUDAGraph() if graph else None
    if graph:
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            step()
    o_lens, o_table, o_free = [0] * n_seq, table.cpu().numpy(), free.tolist()
    o_k, o_v = {}, {}                                              # what the oracle knows to lie at a slot
    for n, change in enumerate([[20, 1, 0, 15], [1, 1, 1, 1], [9, 9, 9, 9], [-5, -8, -9, -2], [1, 0, 20, 1], [-16, 16, 0, -17], [1, 1, 1, 1]]):
        by.copy_(i32(change))
        qkv.copy_(normal(100 + n, n_rows, hq + 2 * hk, d))
        last.copy_(normal(200 + n, n_seq, hq, d))
        was = qkv.clone()
        torch.cuda.synchronize()
        g.replay() if graph else step()
        torch.cuda.synchronize()
        o_lens, o_table, o_free, o_cu, o_pos, o_slots = paged_step.resize(change, o_lens, o_table, o_free, page)
        rows = o_cu[-1]
        assert cu.tolist() == o_cu and positions.tolist() == o_pos + [-1] * (n_rows - rows)
        assert slots.tolist() == o_slots + [-1] * (n_rows - rows)
        assert lens.tolist() == o_lens and np.array_equal(table.cpu().numpy(), o_table)
        assert torch.equal(qkv[rows:], was[rows:]) and torch.equal(v, was[:, hq + hk:])
        freqs = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
        for x, raw in ((q, was[:, :hq]), (k, was[:, hq:hq + hk])):
            ref, size = paged_step.norm_rope(f64(raw[:rows]), f64(gain), 1e-6, o_pos, freqs, False)
            assert (np.abs(f64(x[:rows]) - ref) <= U * np.abs(ref) + 40 * 2.0 ** -24 * size).all()
        for r, slot in enumerate(o_slots):
            for at, x in ((o_k, f64(k[r])), (o_v, f64(v[r]))):
                if dtype == mv.DTYPE_E4M3:
                    x = serving.stored_value(*serving.quantise(x))
                elif dtype == mv.DTYPE_E2M1:
                    code, byte = paged_step.quantise(x)
                    x = paged_step.stored_value(paged_step.pack(code), byte)
                at[slot] = x
        for b, length in enumerate(o_lens):
            at = [int(o_table[b, p // page]) * page + p % page for p in range(length)]
            for h in range(hq):
                kk = np.array([o_k[i][h // 3] for i in at]).reshape(length, d)
                vv = np.array([o_v[i][h // 3] for i in at]).reshape(length, d)
                ref, mag = serving.attend(f64(last[b, h:h + 1]), kk, vv, 0.125, np.ones((1, length), dtype=bool))
                s = (d + 8) * 2.0 ** -23 * 0.125 * np.max(np.abs(f64(last[b, h])) @ np.abs(kk).T, initial=0.0)
                tol = U * np.abs(ref) + (U + 2 * s + (length + 8) * 2.0 ** -23) * mag + 1e-30
                assert (np.abs(f64(out[b, h:h + 1]) - ref) <= tol).all()
