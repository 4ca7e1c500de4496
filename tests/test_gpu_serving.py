"""GPU parity of the serving operators (packed prompt attention, paged cache rows, paged attention) with the oracle.

Tolerances. What a cache holds is compared bit for bit. An attention's element may be off its float64 value by
  u |ref|                the result's rounding to bf16, u = 2^-8 of its magnitude at most (half a step),
  (w + 2 s + n 2^-23) A  with A = sum_j p_j |v_j|: the weights' own rounding w (bf16: 2^-8), the error s of an exponent,
                         (D + 8) 2^-23 scale max_j sum_d |q_d k_jd| for products summed in fp32 plus the rounding of the
                         exponent itself, and fp32 sums over n keys.
"""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import serving

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
BF16, E4M3 = mv.DTYPE_BF16, mv.DTYPE_E4M3


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


def check(got, ref, mag, q, k, scale, keys):
    """Every element within the bound above; q [.., Hq, D], k [.., Hk, D] float64 (their finite entries)."""
    d = q.shape[-1]
    group = q.shape[-2] // k.shape[-2]
    kmax = np.max(np.abs(np.where(np.isfinite(k), k, 0.0)).reshape(-1, k.shape[-2], d), axis=0, initial=0.0)
    dots = scale * np.sum(np.abs(np.where(np.isfinite(q), q, 0.0)) * np.repeat(kmax, group, axis=0), axis=-1)
    s = ((d + 8) * 2.0 ** -23 * dots)[..., None]
    tol = U * np.abs(ref) + (U + 2 * s + (keys + 8) * 2.0 ** -23) * mag + 1e-30
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.array_equal(ref[~fin & ~np.isnan(ref)], got[~fin & ~np.isnan(ref)])
    off = np.abs(got - ref)[fin] / tol[fin]
    assert off.size == 0 or off.max() <= 1.0, f"{off.max():.2f} of the bound"


# ------------------------------------------------------------------------------------------------ prompts

def run_prompt(lens, hq, hk, d, seed=0, scale=None, std=1.0, extra=0):
    t = sum(lens) + extra
    q, k, v = normal(seed, t, hq, d, std=std), normal(seed + 1, t, hk, d, std=std), normal(seed + 2, t, hk, d)
    out = torch.full_like(q, 7.0)
    scale = d ** -0.5 if scale is None else scale
    mv.prompt_attention(q, k, v, mv.PromptPlan(lens, hq // hk), scale, out)
    torch.cuda.synchronize()
    return q, k, v, out, scale


def check_prompt(q, k, v, out, lens, scale):
    n = sum(lens)
    ref, mag = serving.prompt_attention(f64(q)[:n], f64(k)[:n], f64(v)[:n], lens, scale)
    check(f64(out)[:n], ref, mag, f64(q)[:n], f64(k)[:n], scale, max(lens, default=0))


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [256], [257, 1, 64], [0, 5, 0, 300], [640, 33]])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 128), (4, 2, 64)])
def test_prompt_lengths(lens, hq, hk, d):
    q, k, v, out, scale = run_prompt(lens, hq, hk, d)
    check_prompt(q, k, v, out, lens, scale)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (5, 1), (7, 1), (16, 2), (6, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_groups(hq, hk, d):
    lens = [300, 70, 129]
    q, k, v, out, scale = run_prompt(lens, hq, hk, d, seed=hq)
    check_prompt(q, k, v, out, lens, scale)


@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 72, 80, 96, 104, 120])
def test_prompt_head_dims(d):
    lens = [200, 17]
    q, k, v, out, scale = run_prompt(lens, 4, 2, d, seed=d)
    check_prompt(q, k, v, out, lens, scale)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (0.5, 4.0), (1.0, 6.0), (1e-3, 1.0)])
def test_prompt_scales(scale, std):
    """Uniform weights, and scores whose maximum moves by far more than any threshold within a row."""
    lens = [500, 90]
    q, k, v, out, scale = run_prompt(lens, 2, 1, 64, seed=9, scale=scale, std=std)
    check_prompt(q, k, v, out, lens, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,k0", [(1.0, 2.0 ** 20), (0.125, 2.0 ** 9), (1.0, 2.0 ** 40), (0.125, -2.0 ** 20), (2e38, 2.0 ** -110),
                                      (0.0, 2.0 ** 100), (1e-37, 2.0 ** 90)])
def test_scores_of_any_size(d, scale, k0):
    """Scores that fp32 holds exactly, from tiny to larger than 2^24: each is one product, and two keys' differ by nothing
    or by k0 / 8 times 2^20 scale. So a softmax's weights are known to the rounding of an exponent of at most 2^-23 |score|,
    and where the scores differ by more than 2^10 they are 0 and 1; below that here no score is over 2^7."""
    n, hq, hk = 400, 2, 1
    q, k = torch.zeros(n, hq, d, device="cuda"), torch.zeros(n, hk, d, device="cuda")
    q[:, :, 0] = 2.0 ** 20
    k[:, :, 0] = k0 * (1 + (torch.arange(n, device="cuda") * 5 % 7)[:, None] / 8)
    q, k, v = q.to(torch.bfloat16), k.to(torch.bfloat16), normal(3, n, hk, d)
    got = torch.empty_like(q)
    mv.prompt_attention(q, k, v, mv.PromptPlan([n], hq), scale, got)
    pool = Pool([n], hk, d, 16, BF16)
    mv.paged_kv_append(k, v, i32([0, n]), pool.cache, pool.d_table, pool.d_lens)
    one = run_paged(pool, q[-1:].contiguous(), scale)
    scale = float(np.float32(scale))
    top = abs(k0) * 2.0 ** 21 * scale                         # more than any score
    assert top < 2.0 ** 7 or top / 16 > 2.0 ** 10
    ref, mag = serving.prompt_attention(f64(q), f64(k), f64(v), [n], scale)
    tol = U * np.abs(ref) + (U + (top * 2.0 ** -21 if top < 2.0 ** 7 else 0.0) + (n + 8) * 2.0 ** -23) * mag
    assert (np.abs(f64(got) - ref) <= tol).all()
    assert (np.abs(f64(one)[0] - ref[-1]) <= tol[-1]).all()


def test_prompt_rising_scores():
    """Each later key scores higher, so every tile moves the running maximum."""
    n, d = 900, 64
    q = torch.ones(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(n, device="cuda")[:, None, None] * 0.05).expand(n, 1, d).to(torch.bfloat16).contiguous()
    v, out = normal(3, n, 1, d), torch.empty_like(q)
    mv.prompt_attention(q, k, v, mv.PromptPlan([n]), 0.2, out)
    check_prompt(q, k, v, out, [n], 0.2)


def test_prompt_long():
    lens = [2500, 1111]
    q, k, v, out, scale = run_prompt(lens, 2, 1, 128, seed=4)
    check_prompt(q, k, v, out, lens, scale)


@pytest.mark.parametrize("hq,hk", [(8, 8), (12, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_many_items(hq, hk, d):
    """Several times more work items than SMs, of every length up to five key tiles, a NaN in one of the prompts."""
    r = np.random.default_rng(d)
    lens = [int(x) for x in np.concatenate([r.integers(1, 130, 40), r.integers(100, 640, 30), [0, 1, 128, 129, 640]])]
    q, k, v, out, scale = run_prompt(lens, hq, hk, d, seed=d)
    check_prompt(q, k, v, out, lens, scale)
    at = sum(lens[:50]) + lens[50] // 2
    v[at, 0, 5] = float("nan")
    bad = torch.empty_like(out)
    mv.prompt_attention(q, k, v, mv.PromptPlan(lens, hq // hk), scale, bad)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[at:sum(lens[:51]), : hq // hk, 5] = True
    assert torch.equal(bad[~hit], out[~hit]) and torch.isnan(bad[hit]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_of_many_items_at_once(d):
    """Calls that each fill the GPU several times over, on streams of both priorities and replayed from a graph beside them,
    give what each gives alone: a CTA takes over further items of its own call only, each item once."""
    cases = []
    for seed, (n, most, hq, hk) in enumerate([(60, 400, 8, 8), (9, 2000, 8, 2), (150, 130, 12, 4)]):
        lens = [int(x) for x in np.random.default_rng(seed).integers(1, most, n)]
        q, k, v, want, scale = run_prompt(lens, hq, hk, d, seed=seed)
        plan = mv.PromptPlan(lens, hq // hk)
        cases.append((q, k, v, plan, scale, want, torch.empty_like(want), torch.cuda.Stream(priority=-(seed % 2))))
    g, graphed = torch.cuda.CUDAGraph(), torch.zeros_like(cases[0][5])
    with torch.cuda.graph(g):
        for _ in range(2):
            mv.prompt_attention(*cases[0][:5], graphed)
    torch.cuda.synchronize()
    for _ in range(3):
        for q, k, v, plan, scale, _, out, stream in cases:
            mv.prompt_attention(q, k, v, plan, scale, out, stream=stream)
        g.replay()
    torch.cuda.synchronize()
    for *_, want, out, _ in cases:
        assert torch.equal(out, want)
    assert torch.equal(graphed, cases[0][5])


@pytest.mark.parametrize("d", [16, 64, 128])
def test_prompt_rows_repeat_while_their_maximum_moves(d):
    """Both threads of a row use the maximum of the same tile: scores that rise by more than any threshold from tile to
    tile, in more items than SMs, give the same bits on every call, beside another call that disturbs the timing too."""
    lens, hq, hk = [1500, 1, 900, 1100, 640], 8, 4
    t = sum(lens)
    q = (normal(1, t, hq, d).abs() + 0.5).to(torch.bfloat16)
    at = torch.cat([torch.arange(n) for n in lens]).cuda()[:, None, None]
    k = ((at * (0.12 / d) + 0.05 * normal(2, t, hk, d).float()) * d ** 0.5).to(torch.bfloat16)
    v, plan, scale = normal(3, t, hk, d), mv.PromptPlan(lens, hq // hk), 1.0
    first = torch.empty_like(q)
    mv.prompt_attention(q, k, v, plan, scale, first)
    check_prompt(q, k, v, first, lens, scale)
    side, outs, other = torch.cuda.Stream(), [torch.full_like(q, 7.0) for _ in range(24)], torch.empty_like(q)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        mv.prompt_attention(q, k, v, plan, scale, out)
        if i % 2:
            mv.prompt_attention(q, k, v, plan, 0.1, other, stream=side)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, first)


@pytest.mark.parametrize("d", [64, 128])
def test_every_call_of_many_at_once_is_done_in_full(d):
    """Prompt and paged attention on four streams and from a graph with two calls, each call into rows of its own that held a
    NaN before: what a call leaves out stays to be seen."""
    nan, jobs = float("nan"), []
    for seed, (n, most, hq, hk) in enumerate([(60, 400, 8, 8), (9, 2000, 8, 2), (150, 130, 12, 4)]):
        lens = [int(x) for x in np.random.default_rng(seed).integers(1, most, n)]
        q, k, v, want, scale = run_prompt(lens, hq, hk, d, seed=seed)
        plan, outs = mv.PromptPlan(lens, hq // hk), [torch.full_like(want, nan) for _ in range(6)]
        jobs.append((want, outs, torch.cuda.Stream(priority=-(seed % 2)),
                     lambda out, stream=None, a=(q, k, v, plan, scale): mv.prompt_attention(*a, out, stream=stream)))
    for lens, hq, hk, dtype in (([3000, 5], 8, 2, E4M3), ([2000], 32, 32, BF16), ([900] * 7 + [0], 6, 2, BF16)):
        pool = Pool(lens, hk, d, 16, dtype).fill(len(lens))
        q = normal(3, len(lens), hq, d)
        ws = torch.zeros(mv.paged_attention_workspace(len(lens), hq, hk, d), dtype=torch.uint8, device="cuda")
        want = run_paged(pool, q, 0.1, ws=ws)
        jobs.append((want, [torch.full_like(want, nan) for _ in range(6)], torch.cuda.Stream(),
                     lambda out, stream=None, a=(q, pool.cache, pool.d_table, pool.d_lens, 0.1), ws=ws:
                     mv.paged_attention(*a, out, ws, stream=stream)))
    g, graphed = torch.cuda.CUDAGraph(), [torch.full_like(jobs[0][0], nan) for _ in range(2)]
    with torch.cuda.graph(g):
        for out in graphed:
            jobs[0][3](out)
    seen = []
    torch.cuda.synchronize()
    for i in range(6):
        for _, outs, stream, call in jobs:
            call(outs[i], stream)
        g.replay()
        seen.append([out.clone() for out in graphed])
        for out in graphed:
            out.fill_(nan)
    torch.cuda.synchronize()
    for want, outs, _, _ in jobs:
        for out in outs:
            assert torch.equal(out, want)
    for outs in seen:
        for out in outs:
            assert torch.equal(out, jobs[0][0])


def test_prompt_leaves_rows_behind_the_plan():
    lens = [130, 20]
    q, k, v, out, scale = run_prompt(lens, 2, 2, 64, extra=45)
    check_prompt(q, k, v, out, lens, scale)
    assert (out[150:] == 7.0).all()


@pytest.mark.parametrize("layout", ["fused_qkv", "head_major"])
def test_prompt_strides(layout):
    lens, hq, hk, d = [190, 61], 4, 2, 64
    n = sum(lens)
    if layout == "fused_qkv":
        x = normal(1, n, hq + 2 * hk, d)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        out = torch.full((n, hq + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        dst = out[:, :hq]
    else:
        q, k, v = (normal(i, h, n + 9, d)[:, :n].transpose(0, 1) for i, h in ((1, hq), (2, hk), (3, hk)))
        out = torch.full((hq, n + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        dst = out[:, :n].transpose(0, 1)
    mv.prompt_attention(q, k, v, mv.PromptPlan(lens, hq // hk), 0.125, dst)
    check_prompt(q, k, v, dst, lens, 0.125)
    assert (out[:, hq:] == 7.0).all() if layout == "fused_qkv" else (out[:, n:] == 7.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 100, 131, 299])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_masked_places_hold_anything(bad, at, d):
    """A NaN or infinity in one token's v (and k) leaves the rows before it and the other prompts as they were."""
    lens, hq, hk = [150, 300, 40], 4, 2
    n = sum(lens)
    q, k, v = normal(1, n, hq, d), normal(2, n, hk, d), normal(3, n, hk, d)
    plan = mv.PromptPlan(lens, 2)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    mv.prompt_attention(q, k, v, plan, 0.125, clean)
    v2, k2 = v.clone(), k.clone()
    v2[150 + at, 1, 3] = bad
    mv.prompt_attention(q, k, v2, plan, 0.125, out)
    torch.cuda.synchronize()
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[150 + at:450, 2:, 3] = True                           # the rows that see it, their heads, its element
    assert torch.equal(out[~hit], clean[~hit])
    assert not torch.isfinite(out[hit]).any()
    ref, _ = serving.prompt_attention(f64(q), f64(k), f64(v2), lens, 0.125)
    fin = np.isfinite(ref)
    assert np.array_equal(fin, ~hit.cpu().numpy())
    assert np.array_equal(np.isnan(ref), torch.isnan(out).cpu().numpy())
    k2[150 + at, 0, 0] = bad
    mv.prompt_attention(q, k2, v, plan, 0.125, out)
    torch.cuda.synchronize()
    keep = torch.ones_like(hit)
    keep[150 + at:450, :2] = False
    assert torch.equal(out[keep], clean[keep])


def test_prompt_rows_do_not_depend_on_the_pack():
    lens, hq, hk, d = [200, 77, 400], 4, 1, 128
    q, k, v, out, scale = run_prompt(lens, hq, hk, d, seed=5)
    t = 0
    for n in lens:
        alone = torch.empty_like(out[t:t + n])
        mv.prompt_attention(q[t:t + n], k[t:t + n], v[t:t + n], mv.PromptPlan([n], hq // hk), scale, alone)
        assert torch.equal(alone, out[t:t + n])
        t += n


def test_prompt_captured_and_on_another_stream():
    lens, hq, hk, d = [260, 33], 2, 1, 64
    q, k, v, out, scale = run_prompt(lens, hq, hk, d, seed=6)
    plan, got = mv.PromptPlan(lens, 2), torch.zeros_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mv.prompt_attention(q, k, v, plan, scale, got, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mv.prompt_attention(q, k, v, plan, scale, got)
    got.zero_()
    q.copy_(normal(60, *q.shape))
    g.replay()
    torch.cuda.synchronize()
    check_prompt(q, k, v, got, lens, scale)


def test_prompt_on_another_stream_right_after_its_plan():
    """A plan's first call may be on any stream: nothing waits between the two here, for plans of ever other lengths."""
    hq, hk, d, cases, side = 4, 2, 64, [], torch.cuda.Stream()
    for i in range(40):
        lens = [int(x) for x in np.random.default_rng(i).integers(0, 500, 1 + 4 * (i % 20))]
        q, k, v = normal(i, sum(lens), hq, d), normal(i + 1, sum(lens), hk, d), normal(i + 2, sum(lens), hk, d)
        cases.append((lens, q, k, v, torch.full_like(q, 7.0)))
    torch.cuda.synchronize()
    plans = []
    for lens, q, k, v, out in cases:
        plans.append(mv.PromptPlan(lens, hq // hk))
        mv.prompt_attention(q, k, v, plans[-1], 0.125, out, stream=side)
    torch.cuda.synchronize()
    for plan, (lens, q, k, v, out) in zip(plans, cases):
        again = torch.full_like(out, 7.0)
        mv.prompt_attention(q, k, v, plan, 0.125, again)
        assert torch.equal(out, again)
    check_prompt(q, k, v, out, lens, 0.125)


def test_prompt_of_no_tokens():
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    mv.prompt_attention(e, e, e, mv.PromptPlan([0, 0]), 1.0, torch.empty_like(e))
    mv.prompt_attention(e, e, e, mv.PromptPlan([]), 1.0, torch.empty_like(e))


# ------------------------------------------------------------------------------------------------ paged rows

class Pool:
    """A paged cache with shuffled pages, sequences of ``lens`` rows and spare table columns that name no page."""

    def __init__(self, lens, hk, d, page, dtype, seed=0, spare=2):
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.lens, self.page, self.dtype, n_pages = list(lens), page, dtype, sum(need) + 3
        order, at = r.permutation(n_pages), 0
        self.table = np.full((len(lens), max(need, default=0) + spare), -77)
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.cache = mv.PagedKV.zeros(n_pages, page, hk, d, dtype)
        self.d_table, self.d_lens = i32(self.table), i32(lens)

    def fill(self, seed, std=1.0):
        """Every row of the pool random, rows of very different sizes; values() are what they stand for."""
        c = self.cache
        for x, e, s in ((c.k, c.k_exp, seed), (c.v, c.v_exp, seed + 1)):
            rows = normal(s, *x.shape, std=std) * torch.exp(normal(s + 50, *x.shape[:3], 1).float()).to(torch.bfloat16)
            if self.dtype == BF16:
                x.copy_(rows)
            else:
                q, ex = serving.quantise(f64(rows))
                x.view(torch.uint8).copy_(torch.as_tensor(q))
                e.copy_(torch.as_tensor(ex))
        return self

    def values(self):
        c = self.cache
        if self.dtype == BF16:
            return f64(c.k), f64(c.v)
        return tuple(serving.stored_value(x.view(torch.uint8).cpu().numpy(), e.cpu().numpy())
                     for x, e in ((c.k, c.k_exp), (c.v, c.v_exp)))

    def bits(self):
        c = self.cache
        return [t.view(torch.uint8).clone() for t in (c.k, c.v, c.k_exp, c.v_exp) if t is not None]


def same_bits(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def rows_like_a_model(seed, *shape):
    """Rows of very different sizes, some all zero, some tiny, some near the type's limits."""
    x = normal(seed, *shape).float() * torch.exp2(normal(seed + 1, *shape[:-1], 1).float() * 6)
    x[::7, 0] = 0.0
    x[3::11, -1] *= 2.0 ** -110
    x[5::13, 0] *= 2.0 ** 100
    x[:, :, 1::5] *= 0.01
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("hk,d,page,lens,rows", [
    (2, 128, 16, [5, 40, 16], [5, 40, 16]), (1, 64, 32, [33, 1, 0, 70], [1, 1, 0, 1]), (3, 16, 48, [100, 7], [55, 0]),
    (5, 80, 16, [31], [17]), (8, 128, 64, [500, 64, 65], [500, 64, 65]), (2, 32, 1024, [1030, 9], [1030, 9]),
    (1, 112, 256, [300], [299])])
def test_append_and_read_back(dtype, hk, d, page, lens, rows):
    pool = Pool(lens, hk, d, page, dtype)
    before = pool.bits()
    cu = np.concatenate([[0], np.cumsum(rows)])
    n = int(cu[-1]) + 6                                       # padded rows behind the last sequence
    k, v = rows_like_a_model(1, n, hk, d), rows_like_a_model(9, n, hk, d)
    mv.paged_kv_append(k, v, i32(cu), pool.cache, pool.d_table, pool.d_lens)
    torch.cuda.synchronize()
    want = [x.cpu().numpy().copy() for x in before]
    for plane, x in enumerate((k, v)):
        if dtype == E4M3:
            q, e = serving.quantise(f64(x))
        else:
            q = x.view(torch.uint8).cpu().numpy()
        for b in range(len(lens)):
            for i in range(rows[b]):
                pos = lens[b] - rows[b] + i
                at = pool.table[b, pos // page], slice(None), pos % page
                want[plane][at] = q[cu[b] + i]
                if dtype == E4M3:
                    want[2 + plane][at] = e[cu[b] + i]
    assert same_bits(pool.bits(), [torch.as_tensor(w).cuda() for w in want])
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32(cu), ko, vo)
    torch.cuda.synchronize()
    for x, y in ((k, ko), (v, vo)):
        assert (y[cu[-1]:] == 7.0).all()
        ref = f64(x)[:cu[-1]]
        if dtype == E4M3:
            ref = serving.stored_value(*serving.quantise(ref))
        with np.errstate(over="ignore"):
            ref = torch.as_tensor(ref.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(y[:cu[-1]].cpu(), ref)


def test_append_nan_and_infinity():
    d = 64
    x = torch.zeros(4, 1, d, dtype=torch.bfloat16, device="cuda")
    x[:, 0, 0] = torch.tensor([1.0, float("nan"), float("inf"), -float("inf")])
    x[:, 0, 1] = 3.0
    pool = Pool([4], 1, d, 16, E4M3)
    out = torch.empty_like(x)
    mv.paged_kv_append(x, x, i32([0, 4]), pool.cache, pool.d_table, pool.d_lens)
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32([0, 4]), out, torch.empty_like(x))
    got = out[:, 0].float().cpu()
    assert got[0, 0] == 1.0 and torch.isnan(got[1, 0]) and got[2, 0] == float("inf") and got[3, 0] == -float("inf")
    assert got[:2, 1].tolist() == [3.0, 3.0]                  # a NaN leaves its row's other values alone
    assert (got[:, 2:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_rows_with_strides_into_a_session_layout(dtype):
    """Written from and read into [H][S][D] planes, the layout of a session's cache."""
    hk, d, n = 4, 64, 90
    pool = Pool([n], hk, d, 32, dtype)
    src = normal(1, 2, hk, 128, d)
    dst = torch.full_like(src, 7.0)
    k, v = (src[c, :, 20:20 + n].transpose(0, 1) for c in range(2))
    ko, vo = (dst[c, :, 3:3 + n].transpose(0, 1) for c in range(2))
    mv.paged_kv_append(k, v, i32([0, n]), pool.cache, pool.d_table, pool.d_lens)
    mv.paged_kv_read(pool.cache, pool.d_table, pool.d_lens, i32([0, n]), ko, vo)
    torch.cuda.synchronize()
    assert (dst[:, :, :3] == 7.0).all() and (dst[:, :, 3 + n:] == 7.0).all()
    for x, y in ((k, ko), (v, vo)):
        want = f64(x) if dtype == BF16 else serving.stored_value(*serving.quantise(f64(x)))
        assert np.array_equal(f64(y), want)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d", [16, 48, 64, 80, 128])
@pytest.mark.parametrize("off", ["k", "v", "heads", "tokens", "pool"])
def test_rows_on_any_multiple_of_16_bytes(dtype, d, off):
    """Rows of the caller's or of the pool that start on odd multiples of 16 bytes move like those on multiples of 32."""
    lens, hk, page = [37, 1, 70], 3, 16
    n, cu = sum(lens), i32(np.cumsum([0] + lens))
    aligned = Pool(lens, hk, d, page, dtype, seed=d)
    k, v = normal(1, n, hk, d), normal(2, n, hk, d)
    mv.paged_kv_append(k, v, cu, aligned.cache, aligned.d_table, aligned.d_lens)

    def rows(which):
        """[n, hk, d] in memory filled with 7, moved by 8 elements where asked"""
        skip, gap_h, gap_t = 8 * (off == which), 8 * (off == "heads"), 8 * (off == "tokens")
        ts = hk * (d + gap_h) + gap_t
        flat = torch.full((skip + n * ts,), 7.0, dtype=torch.bfloat16, device="cuda")
        return flat, flat.as_strided((n, hk, d), (ts, d + gap_h, 1), skip)

    pool = Pool(lens, hk, d, page, dtype, seed=d)
    c = pool.cache
    if off == "pool":
        def moved(x):
            by = 16 // x.element_size()
            return torch.zeros(x.numel() + by, dtype=torch.uint8 if dtype == E4M3 else x.dtype,
                               device="cuda").view(x.dtype)[by:].view(x.shape)
        c = mv.PagedKV(moved(c.k), moved(c.v), c.k_exp, c.v_exp)
        pool.cache = c
    (_, k1), (_, v1) = rows("k"), rows("v")
    k1.copy_(k)
    v1.copy_(v)
    mv.paged_kv_append(k1, v1, cu, c, pool.d_table, pool.d_lens)
    assert same_bits(pool.bits(), aligned.bits())
    (fk, ko), (fv, vo) = rows("k"), rows("v")
    want = [torch.empty_like(k) for _ in range(2)]
    mv.paged_kv_read(aligned.cache, aligned.d_table, aligned.d_lens, cu, *want)
    mv.paged_kv_read(c, pool.d_table, pool.d_lens, cu, ko, vo)
    torch.cuda.synchronize()
    for x, src, flat, got in ((want[0], k, fk, ko), (want[1], v, fv, vo)):
        assert torch.equal(got, x)
        ref = f64(src) if dtype == BF16 else serving.stored_value(*serving.quantise(f64(src)))
        assert np.array_equal(f64(x), ref)
        got.fill_(7.0)
        assert (flat == 7.0).all()                            # nothing between the rows


def take_error(site):
    st, code = mv.get_error()
    assert st == 6 and code >> 16 == site and code & 0xffff == 2


@pytest.mark.parametrize("what", ["page_high", "page_low", "len_high", "len_negative", "too_many_rows", "cu_falls",
                                  "cu_past_rows", "cu_first"])
def test_rows_out_of_range_are_reported_and_left_alone(what):
    hk, d, page = 2, 64, 16
    pool = Pool([20, 40], hk, d, page, E4M3, spare=0)
    table, lens, cu = pool.table.copy(), [20, 40], [0, 20, 60]
    if what == "page_high":
        table[1, 1] = pool.cache.n_pages
    elif what == "page_low":
        table[1, 1] = -1
    elif what == "len_high":
        lens[1] = 49                                          # three pages of 16 in the table's row
    elif what == "len_negative":
        lens[1] = -5
    elif what == "too_many_rows":
        lens[1] = 39
    elif what == "cu_falls":
        cu = [0, 20, 5]
    elif what == "cu_past_rows":
        cu = [0, 20, 61]
        lens[1] = 41
    elif what == "cu_first":
        cu = [3, 20, 60]
        lens[0] = 17
    x = normal(1, 60, hk, d)
    before = pool.bits()
    mv.paged_kv_append(x, x, i32(cu), pool.cache, i32(table), i32(lens))
    take_error(40)
    changed = [(a != b) for a, b in zip(pool.bits(), before)]
    legal = set(int(p) for p in pool.table.ravel() if p >= 0)
    for c in changed:                                         # nothing outside the sequences' own pages
        rest = [p for p in range(pool.cache.n_pages) if p not in legal]
        assert not c[rest].any()
    out = torch.full_like(x, 7.0)
    mv.paged_kv_read(pool.cache, i32(table), i32(lens), i32(cu), out, out.clone())
    take_error(40)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("what", ["len_high", "len_negative", "too_many_rows", "page_high", "page_low"])
def test_rows_of_a_bad_sequence_or_page_stay_where_they_are(dtype, what):
    """Neither written nor read back: all rows of a sequence with a bad length, the rows of a bad page; the others move."""
    hk, d, page, rows = 2, 64, 16, [20, 30, 25]
    lens = [20, 48, 25]                                       # three pages of 16 in the table's rows
    pool = Pool(lens, hk, d, page, dtype, spare=0)
    cu, table, cur = i32(np.cumsum([0] + rows)), pool.table.copy(), list(lens)
    left_out = list(range(20, 50))
    if what == "len_high":
        cur[1] = 60                                           # the first 18 of its rows would have places below 48
    elif what == "len_negative":
        cur[1] = -1
    elif what == "too_many_rows":
        cur[1] = 29
    else:
        table[1, 1] = pool.cache.n_pages if what == "page_high" else -1   # positions 16 .. 31: rows 20 .. 33
        left_out = list(range(20, 34))
    x, y = normal(1, sum(rows), hk, d), normal(2, sum(rows), hk, d)
    keep = [i for i in range(sum(rows)) if i not in left_out]
    before = pool.bits()
    mv.paged_kv_append(x, y, cu, pool.cache, i32(table), i32(cur))
    take_error(40)
    after = pool.bits()
    mv.paged_kv_append(x, y, cu, pool.cache, pool.d_table, i32(lens))     # what the pool holds with all rows
    full = pool.bits()
    at = [(int(pool.table[b, p // page]), p % page) for b in range(3) for p in range(lens[b] - rows[b], lens[b])]
    for was, now, whole in zip(before, after, full):
        want = was.clone()
        for i in keep:
            want[at[i][0], :, at[i][1]] = whole[at[i][0], :, at[i][1]]
        assert torch.equal(now, want)
    want, got = ([torch.full_like(x, 7.0) for _ in range(2)] for _ in range(2))
    mv.paged_kv_read(pool.cache, pool.d_table, i32(lens), cu, *want)
    mv.paged_kv_read(pool.cache, i32(table), i32(cur), cu, *got)
    take_error(40)
    for w, g in zip(want, got):
        assert torch.equal(g[keep], w[keep]) and (g[left_out] == 7.0).all()


# ------------------------------------------------------------------------------------------------ paged attention

def run_paged(pool, q, scale, table=None, lens=None, ws=None):
    b, hq, d = q.shape
    if ws is None:
        ws = torch.zeros(mv.paged_attention_workspace(b, hq, pool.cache.n_kv_heads, d), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    mv.paged_attention(q, pool.cache, pool.d_table if table is None else table, pool.d_lens if lens is None else lens,
                       scale, out, ws)
    torch.cuda.synchronize()
    return out


def check_paged(pool, q, out, scale, lens=None):
    lens = pool.lens if lens is None else lens
    kp, vp = pool.values()
    ref, mag = serving.paged_attention(f64(q), kp, vp, pool.table, lens, scale)
    got = f64(out)
    for b, n in enumerate(lens):
        k = serving.sequence_rows(kp, pool.table[b], n)
        check(got[b:b + 1], ref[b:b + 1], mag[b:b + 1], f64(q)[b:b + 1], k, scale, n)


LENS = [[1], [0], [16, 15, 17, 0, 1], [127, 128, 129, 255, 257], [700, 3], [1], [64] * 9]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("hq,hk,d,page", [(8, 2, 128, 16), (4, 4, 64, 32)])
def test_paged_attention_lengths(dtype, lens, hq, hk, d, page):
    pool = Pool(lens, hk, d, page, dtype).fill(1)
    q = normal(3, len(lens), hq, d)
    out = run_paged(pool, q, d ** -0.5)
    check_paged(pool, q, out, d ** -0.5)
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (7, 1), (8, 1), (9, 1), (10, 2), (16, 1), (17, 1), (40, 2), (33, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_attention_groups(dtype, hq, hk, d):
    lens = [200, 35]
    pool = Pool(lens, hk, d, 16, dtype).fill(hq)
    q = normal(3, len(lens), hq, d)
    check_paged(pool, q, run_paged(pool, q, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d", [16, 32, 48, 80, 96, 112])
@pytest.mark.parametrize("page", [16, 48, 1024])
def test_paged_attention_head_dims_and_pages(dtype, d, page):
    lens = [333, 48, 49]
    pool = Pool(lens, 2, d, page, dtype).fill(d)
    q = normal(3, len(lens), 6, d)
    check_paged(pool, q, run_paged(pool, q, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_paged_attention_long_and_many(dtype):
    """One sequence long enough to be split over the whole GPU, and more sequences than SMs."""
    pool = Pool([9001, 2], 1, 64, 64, dtype).fill(1)
    q = normal(3, 2, 4, 64)
    check_paged(pool, q, run_paged(pool, q, 0.125), 0.125)
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 300, 400)]
    pool = Pool(lens, 2, 64, 16, dtype).fill(1)
    q = normal(3, len(lens), 4, 64)
    check_paged(pool, q, run_paged(pool, q, 0.125), 0.125)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n_seq", [1025, 2500])
def test_paged_attention_of_more_sequences_than_a_launch_takes(dtype, n_seq):
    lens = [int(x) for x in np.random.default_rng(n_seq).integers(0, 40, n_seq)]
    pool = Pool(lens, 1, 32, 16, dtype).fill(1)
    q = normal(3, n_seq, 2, 32)
    out = run_paged(pool, q, 0.2)
    check_paged(pool, q, out, 0.2)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("hq,hk,d,page,lens", [
    (16, 8, 128, 64, [9001, 7310, 0, 8800, 5, 9999, 6007, 8191]),      # 8 kv heads, units of some 70 steps (bf16)
    (8, 8, 64, 16, [30011, 31, 28000, 160, 30500, 25001]),             # steps of 256 (512) keys
    (20, 2, 128, 32, [33000, 700, 31017, 1, 29999, 20011, 26000, 30])])  # two tiles of heads a unit
def test_paged_attention_of_long_pieces(dtype, hq, hk, d, page, lens):
    """Pieces of more than 20 places, spread over all CTAs with some one longer, units cut into parts at any step and also
    between their start and first step: a CTA's piece is total / 152 = 21 to 35 places, a unit's width n / step + 2."""
    steps = {(BF16, 128): 128, (BF16, 64): 256, (E4M3, 128): 256, (E4M3, 64): 512}[dtype, d]
    total = sum(hk * (2 + max(1, -(-n // steps))) for n in lens)
    while total <= 21 * 152:                                  # 8-bit caches: as many sequences as that takes
        total += sum(hk * (2 + max(1, -(-n // steps))) for n in lens)
        lens = lens + lens
    pool = Pool(lens, hk, d, page, dtype)
    k, v = (normal(i, sum(lens), hk, d) * torch.exp2(normal(i + 9, sum(lens), hk, 1)) for i in (1, 2))
    mv.paged_kv_append(k, v, i32(np.cumsum([0] + lens)), pool.cache, pool.d_table, pool.d_lens)
    q = normal(3, len(lens), hq, d)
    ws = torch.zeros(mv.paged_attention_workspace(len(lens), hq, hk, d), dtype=torch.uint8, device="cuda")
    out = run_paged(pool, q, d ** -0.5, ws=ws)
    assert torch.equal(run_paged(pool, q, d ** -0.5, ws=ws), out)
    for b, n in enumerate(lens[:8]):                          # every sequence's first, some of its further kv heads
        if n == 0:
            assert (out[b] == 0).all()
            continue
        ids = torch.as_tensor(pool.table[b, : -(-n // page)], device="cuda").long()
        for c in sorted({0, b % hk, hk - 1}):
            rows, heads = [], slice(c * (hq // hk), (c + 1) * (hq // hk))
            for x, e in ((pool.cache.k, pool.cache.k_exp), (pool.cache.v, pool.cache.v_exp)):
                r = (x.view(torch.uint8)[ids, c].view(x.dtype) if dtype == E4M3 else x[ids, c]).float().double()
                if dtype == E4M3:
                    r = r * torch.exp2(e[ids, c].double() - 127)[..., None]
                rows.append(r.reshape(-1, d)[:n].cpu().numpy())
            one = f64(q[b, heads])
            ref, mag = serving.attend(one, *rows, d ** -0.5, np.ones((len(one), n), dtype=bool))
            check(f64(out[b, heads]), ref, mag, one, rows[0][:, None], d ** -0.5, n)


@pytest.mark.parametrize("dtype,cols", [(BF16, 1027), (E4M3, 2060)])
def test_paged_attention_of_wide_tables(dtype, cols):
    """1024 sequences of 256 kv heads under a table for a million positions each: more places on the line than 31 bits count
    if all were in use, so it takes several launches. The sequences share their pages and are short."""
    n_seq, hk, d, page = 1024, 256, 128, 1024
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 40, n_seq)]
    lens[3], lens[1021] = 900, 700
    cache = mv.PagedKV.zeros(2, page, hk, d, dtype)
    k, v = normal(1, page, hk, d), normal(2, page, hk, d)
    mv.paged_kv_append(k, v, i32([0, page]), cache, i32([[1]]), i32([page]))
    held = [torch.empty_like(k) for _ in range(2)]
    mv.paged_kv_read(cache, i32([[1]]), i32([page]), i32([0, page]), *held)
    table = torch.full((n_seq, cols), -5, dtype=torch.int32, device="cuda")
    table[:, 0] = 1
    q = normal(3, n_seq, hk, d)
    ws = torch.zeros(mv.paged_attention_workspace(n_seq, hk, hk, d), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    mv.paged_attention(q, cache, table, i32(lens), 0.1, out, ws)
    torch.cuda.synchronize()
    for b in (0, 3, 500, 1010, 1018, 1019, 1020, 1021, 1023):
        for h in (0, 101, 255):
            n = lens[b]
            one = f64(q[b:b + 1, h:h + 1])
            ks, vs = (f64(x[:n, h]) for x in held)
            ref, mag = serving.attend(one[:, 0], ks, vs, 0.1, np.ones((1, n), dtype=bool))
            check(f64(out[b:b + 1, h]), ref, mag, one[0], ks[:, None], 0.1, n)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n", [0, 1, 15, 130, 1000, 2300])
@pytest.mark.parametrize("hq,hk,d", [(32, 32, 128), (64, 8, 64), (16, 8, 128), (128, 128, 64), (64, 64, 32), (144, 9, 128)])
def test_paged_attention_of_one_sequence(dtype, n, hq, hk, d):
    """One sequence over one to sixteen CTAs for each unit, with fewer steps than CTAs among them."""
    pool = Pool([n], hk, d, 48, dtype).fill(n)
    q = normal(3, 1, hq, d)
    out = run_paged(pool, q, d ** -0.5)
    check_paged(pool, q, out, d ** -0.5)
    assert n or (out == 0).all()
    if n == 1000:                                             # captured, replayed at another length
        ws = torch.zeros(mv.paged_attention_workspace(1, hq, hk, d), dtype=torch.uint8, device="cuda")
        g, got, cur = torch.cuda.CUDAGraph(), torch.empty_like(q), i32([1])
        with torch.cuda.graph(g):
            mv.paged_attention(q, pool.cache, pool.d_table, cur, d ** -0.5, got, ws)
        cur.fill_(n)
        g.replay()
        assert torch.equal(got, out)
    if n == 130:
        bad = run_paged(pool, q, 0.1, lens=i32([-1]))
        take_error(41)
        assert (bad == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (1.0, 3.0)])
def test_paged_attention_scales(dtype, scale, std):
    pool = Pool([400, 50], 2, 64, 16, dtype).fill(1, std)
    q = normal(3, 2, 6, 64, std=std)
    check_paged(pool, q, run_paged(pool, q, scale), scale)


def test_paged_attention_value_rows_of_any_size():
    """Value rows whose scales lie far apart, a row of zeros under the largest weight among them."""
    n, d = 64, 64
    k = normal(1, n, 1, d, std=0.1)
    v = (normal(2, n, 1, d).float() * torch.exp2(torch.linspace(-60, 40, n, device="cuda"))[:, None, None])
    q = normal(3, 1, 2, d)
    k[5], v[5] = q[0, :1] * 3, 0.0
    v = v.to(torch.bfloat16)
    pool = Pool([n], 1, d, 16, E4M3)
    mv.paged_kv_append(k, v, i32([0, n]), pool.cache, pool.d_table, pool.d_lens)
    out = run_paged(pool, q, 1.0)
    check_paged(pool, q, out, 1.0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,hq,d,n_seq", [(64, 2, 64, 1), (900, 8, 128, 2), (40, 12, 128, 300), (2500, 3, 64, 3)])
def test_paged_attention_of_columns_that_few_rows_fill(dtype, n, hq, d, n_seq):
    """Every column's value comes from its own rows, however far their sizes and weights lie below those of rows that have
    nothing there: each value row fills one column in 16, its size and its key's score follow the column."""
    rows = np.arange(n_seq * n)
    col = rows % 16
    size = 2.0 ** (12.0 * (col - 8))                          # 2^-96 .. 2^84
    v = np.zeros((len(rows), 1, d))
    fill = np.abs(f64(normal(1, len(rows), 1, d))) + 0.25
    v[:, 0, :] = np.where(np.arange(d)[None] % 16 == col[:, None], fill[:, 0] * size[:, None], 0.0)
    k = np.zeros_like(v)
    k[:, 0, 0] = -2.5 * (col * 7 % 16)                        # weights down to e^-37.5 of the largest
    q = np.zeros((n_seq, hq, d))
    q[:, :, 0] = 1.0 + 0.0625 * (np.arange(hq) % 4)
    k, v, q = (torch.as_tensor(x, device="cuda").to(torch.bfloat16) for x in (k, v, q))
    pool = Pool([n] * n_seq, 1, d, 16, dtype)
    mv.paged_kv_append(k, v, i32(np.arange(n_seq + 1) * n), pool.cache, pool.d_table, pool.d_lens)
    out = run_paged(pool, q, 1.0)
    check_paged(pool, q, out, 1.0)
    # nothing is lost above bf16's normal range (below it, a value may round to zero: column 2 with q = 1.1875 has
    # 2^-72 e^(-2.5 * 14 * 1.1875) 0.25 = 2^-133.96, under half of the smallest bf16)
    ref, _ = serving.paged_attention(f64(q), *pool.values(), pool.table, pool.lens, 1.0)
    assert (f64(out)[ref > 2.0 ** -126] != 0).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [5, 700])
def test_paged_attention_of_nan_and_infinity(dtype, bad, n):
    """In a value row that is attended to: out of its kv head's query heads is not finite there, and the others' as it was."""
    hq, hk, d, at = 6, 2, 64, n // 2
    pool = Pool([n], hk, d, 16, dtype)
    k, v, q = normal(1, n, hk, d), normal(2, n, hk, d), normal(3, 1, hq, d)
    args = i32([0, n]), pool.cache, pool.d_table, pool.d_lens
    mv.paged_kv_append(k, v, *args)
    clean = run_paged(pool, q, 0.125)
    v[at, 1, 7] = bad
    mv.paged_kv_append(k, v, *args)
    out = run_paged(pool, q, 0.125)
    assert torch.equal(out[:, :3], clean[:, :3])
    assert not torch.isfinite(out[:, 3:, 7]).any()
    assert torch.isfinite(out[:, 3:, :7]).all() and torch.isfinite(out[:, 3:, 8:]).all()
    if dtype == BF16 or bad != bad:                           # a NaN does not count for its row's scale
        rest = [e for e in range(d) if e != 7]
        assert torch.equal(out[:, 3:, rest], clean[:, 3:, rest])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n", [1, 13, 16, 100])
def test_paged_attention_ignores_what_lies_behind(dtype, n):
    pool = Pool([n], 2, 128, 64, dtype).fill(1)
    q = normal(3, 1, 8, 128)
    clean = run_paged(pool, q, 0.1)
    c = pool.cache
    for x in (c.k, c.v, c.k_exp, c.v_exp):
        if x is None:
            continue
        raw = x.view(torch.uint8)
        keep = [(int(pool.table[0, p // 64]), p % 64) for p in range(n)]
        junk = torch.full_like(raw, 0x7f) if x.dtype != torch.uint8 else torch.full_like(raw, 0xff)
        for page, slot in keep:
            junk[page, :, slot] = raw[page, :, slot]
        if dtype == BF16:
            junk = torch.where(junk == 0x7f, torch.full_like(junk, 0xff), junk)  # 0xffff: a NaN
            for page, slot in keep:
                junk[page, :, slot] = raw[page, :, slot]
        raw.copy_(junk)
    assert torch.equal(run_paged(pool, q, 0.1), clean)


def test_paged_attention_strides_and_shared_pages():
    """q and out as slices of wider rows; two sequences that share their first pages."""
    pool = Pool([100, 70], 2, 64, 16, BF16).fill(1)
    pool.table[1, :4] = pool.table[0, :4]
    pool.d_table = i32(np.pad(pool.table, ((0, 0), (0, 5)), constant_values=-9))[:, :pool.table.shape[1]]
    x = normal(3, 2, 9, 64)
    q, buf = x[:, 2:6], torch.full((4, 2, 64 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, :64].transpose(0, 1)
    ws = torch.zeros(mv.paged_attention_workspace(2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    mv.paged_attention(q, pool.cache, pool.d_table, pool.d_lens, 0.125, out, ws)
    check_paged(pool, q, out, 0.125)
    assert (buf[:, :, 64:] == 7.0).all()


def test_paged_attention_repeats_bit_for_bit_and_leaves_its_workspace_clean():
    pool = Pool([5000, 3, 800], 2, 128, 16, E4M3).fill(1)
    q = normal(3, 3, 8, 128)
    ws = torch.zeros(mv.paged_attention_workspace(3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    first = run_paged(pool, q, 0.1, ws=ws)
    small = Pool([40], 1, 64, 16, BF16).fill(2)               # another shape through the same workspace in between
    run_paged(small, normal(4, 1, 2, 64), 0.1, ws=ws)
    for _ in range(20):
        assert torch.equal(run_paged(pool, q, 0.1, ws=ws), first)


@pytest.mark.parametrize("what", ["page_high", "page_low", "len_high", "len_negative"])
def test_paged_attention_out_of_range_is_reported(what):
    pool = Pool([200, 40, 30], 2, 64, 16, E4M3, spare=0).fill(1)
    q = normal(3, 3, 4, 64)
    ws = torch.zeros(mv.paged_attention_workspace(3, 4, 2, 64), dtype=torch.uint8, device="cuda")
    good = run_paged(pool, q, 0.1, ws=ws)
    table, lens = pool.table.copy(), list(pool.lens)
    if what == "page_high":
        table[0, 7] = pool.cache.n_pages
    elif what == "page_low":
        table[0, 7] = -1
    elif what == "len_high":
        lens[1] = table.shape[1] * 16 + 1
    else:
        lens[1] = -1
    run_paged(pool, q, 0.1, i32(table), i32(lens), ws)
    take_error(41)
    assert torch.equal(run_paged(pool, q, 0.1, ws=ws), good)  # the workspace serves later calls


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,hq,hk,d", [
    ([40, 17, 300, 0, 90], 4, 2, 64),                         # pieces of the line, units cut across CTAs
    ([100] * 200 + [33], 32, 4, 128),                         # a unit to each warp
    ([700, 64, 900, 128], 48, 4, 128),                        # two tiles of heads a unit
    ([1000], 32, 32, 128), ([1300], 8, 1, 64), ([2300], 96, 8, 64)])   # one sequence: clusters, and pieces
@pytest.mark.parametrize("nth", [0, 1, -1])
@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_paged_attention_leaves_the_row_of_a_bad_page_alone(dtype, lens, hq, hk, d, nth, entry):
    """A page outside the pool: the rows of its sequence are not written, all others are what they are without it."""
    pool = Pool(lens, hk, d, 16, dtype, spare=0).fill(len(lens))
    q = normal(3, len(lens), hq, d)
    ws = torch.zeros(mv.paged_attention_workspace(len(lens), hq, hk, d), dtype=torch.uint8, device="cuda")
    good = run_paged(pool, q, 0.1, ws=ws)
    b = int(np.argmax(lens)) if nth else 0
    table = pool.table.copy()
    table[b, nth % -(-lens[b] // 16)] = entry
    out = run_paged(pool, q, 0.1, i32(table), ws=ws)
    take_error(41)
    rest = [i for i in range(len(lens)) if i != b]
    assert (out[b] == 7.0).all() and torch.equal(out[rest], good[rest])
    lens2 = list(lens)
    lens2[b] = 16 * (nth % -(-lens[b] // 16))                 # the same table, a length that ends before it
    out = run_paged(pool, q, 0.1, i32(table), i32(lens2), ws)
    check_paged(pool, q, out, 0.1, lens2)


def test_paged_attention_of_no_sequences():
    c = mv.PagedKV.zeros(1, 16, 2, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mv.paged_attention_workspace(0, 4, 2, 64), dtype=torch.uint8, device="cuda")
    mv.paged_attention(q, c, i32(np.zeros((0, 3))), i32([]), 1.0, torch.empty_like(q), ws)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, among them both kinds of split, give what they give alone."""
    cases = []
    for lens, hq, hk, dtype in (([3000, 5], 8, 2, E4M3), ([2000], 32, 32, BF16), ([900] * 7, 6, 2, BF16)):
        pool = Pool(lens, hk, 64, 16, dtype).fill(len(lens))
        q = normal(3, len(lens), hq, 64)
        cases.append((pool, q, run_paged(pool, q, 0.1), torch.empty_like(q), torch.zeros(
            mv.paged_attention_workspace(len(lens), hq, hk, 64), dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    lens = [300, 40, 500]
    q, k, v, want, scale = run_prompt(lens, 4, 2, 64, seed=8)
    plan, got, side = mv.PromptPlan(lens, 2), torch.empty_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for pool, x, _, out, ws, stream in cases:
            mv.paged_attention(x, pool.cache, pool.d_table, pool.d_lens, 0.1, out, ws, stream=stream)
        mv.prompt_attention(q, k, v, plan, scale, got, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for _, _, alone, out, _, _ in cases:
        assert torch.equal(out, alone)


def test_decode_loop_captured_once_and_replayed():
    """Prefill, then a captured step (write the new token's row, attend) replayed as the lengths grow in place."""
    lens, hq, hk, d, page, steps = [30, 77], 4, 2, 64, 16, 5
    t, scale = sum(lens), 0.125
    full = [normal(i, 2, 100, h, d) for i, h in ((1, hq), (2, hk), (3, hk))]   # every sequence's whole stream
    pool = Pool([n + steps for n in lens], hk, d, page, BF16)
    cur = i32(lens)
    pack = [torch.cat([x[b, :n] for b, n in enumerate(lens)]) for x in full]
    out = torch.empty_like(pack[0])
    mv.prompt_attention(*pack, mv.PromptPlan(lens, hq // hk), scale, out)
    check_prompt(*pack, out, lens, scale)
    mv.paged_kv_append(pack[1], pack[2], i32(np.cumsum([0] + lens)), pool.cache, pool.d_table, cur)
    q, k, v = (torch.zeros(2, x.shape[2], d, dtype=torch.bfloat16, device="cuda") for x in full)
    o, one = torch.zeros_like(q), i32([0, 1, 2])
    ws = torch.zeros(mv.paged_attention_workspace(2, hq, hk, d), dtype=torch.uint8, device="cuda")
    saved = cur.clone()

    def step():
        cur.add_(1)
        mv.paged_kv_append(k, v, one, pool.cache, pool.d_table, cur)
        mv.paged_attention(q, pool.cache, pool.d_table, cur, scale, o, ws)

    step()                                                    # warm-up; its row is written again by the replay
    cur.copy_(saved)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(steps):
        for x, y in ((q, full[0]), (k, full[1]), (v, full[2])):
            x.copy_(torch.stack([y[b, n + i] for b, n in enumerate(lens)]))
        g.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            m = n + i + 1
            ref, mag = serving.prompt_attention(f64(full[0][b, :m]), f64(full[1][b, :m]), f64(full[2][b, :m]), [m], scale)
            check(f64(o[b:b + 1]), ref[-1:], mag[-1:], f64(q[b:b + 1]), f64(full[1][b, :m]), scale, m)
