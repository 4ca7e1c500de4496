"""One-token attention over pages of every format where scores are large: a later key's score lies a little above those of all
keys before it, and both are so large that fp32 has no place for the score plus what the reference may be outgrown by.

Scores are built to be exact in fp32: with scale = ln 2 in fp32 the exponent's base is 2 (scale log2(e) rounds to 1), all keys
but one score s 1.5 2^e, possibly one unit in the last place more, and one later key scores D more, a multiple of that place.
Products, sums and differences of such numbers are exact, so weights are 1 and 2^D but for the exponential itself.

Tolerances. An element may be off its float64 value by
  2^-8 |ref|                       its rounding to bf16 (half a step),
  (W + 2^-20 + (n + 8) 2^-23) A    with A = sum_j p_j |v_j|: the weights' rounding (W: 2^-16 over bf16 pages, else 2^-11), the
                                   exponential's 2^-22 and fl(ln 2)'s D 3e-9 (in numerator and denominator), sums of n keys.
"""
import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv

pytestmark = pytest.mark.gpu
LN2 = np.float32(np.log(2.0))
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    mv.lib()


def cases():
    """(sign, e, odd, D): D in units of log2, all multiples of the last place of 1.5 2^e."""
    for e in range(21, 29):
        ulp = 2.0 ** (e - 23)
        for d in (7, 8, 9, 12, 14, 15, 16, 17, 18, 20, 24, 32):
            if d % ulp == 0:
                for sign in (1, -1):
                    for odd in (0, 1):
                        yield sign, e, odd, d


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [mv.DTYPE_BF16, mv.DTYPE_E4M3, mv.DTYPE_E2M1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(4, 1), (12, 1), (8, 2)])
@pytest.mark.parametrize("n,late", [(150, 100), (700, 600)])
def test_reference_moves_at_scores_of_any_size(dtype, d, hq, hk, n, late):
    """A sequence for each case, its late key in a later step than the first ones, of a warp to itself or of eight."""
    todo = list(cases())
    n_seq = len(todo)
    assert LN2 * np.float32(1.4426950408889634) == 1.0 and n_seq > 200
    pages = -(-n // PAGE)
    cache = mv.PagedKV.zeros(n_seq * pages, PAGE, hk, d, dtype)
    table, lens = i32(np.arange(n_seq * pages).reshape(n_seq, pages)), i32([n] * n_seq)
    # columns 0, 16, 32 score; beside the last two a 6 that meets a zero of q makes their group's scale 1
    k = torch.zeros(n_seq, n, hk, d, device="cuda")
    k[..., 0], k[..., 32], k[..., 33] = 6144.0, 1.0, 6.0
    k[:, late, :, 16], k[:, late, :, 17] = 1.0, 6.0
    g = torch.Generator(device="cuda")
    g.manual_seed(d + n)
    v = torch.randn(n_seq, n, hk, d, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.zeros(n_seq, hq, d)
    for b, (sign, e, odd, by) in enumerate(todo):
        q[b, :, 0], q[b, :, 16], q[b, :, 32] = sign * 2.0 ** (e - 12), by, odd * 2.0 ** (e - 23)
    q = q.to(torch.bfloat16).cuda()
    cu = i32(np.arange(n_seq + 1) * n)
    rows = [x.to(torch.bfloat16).reshape(n_seq * n, hk, d) for x in (k, v)]
    mv.paged_kv_append(*rows, cu, cache, table, lens)
    ko, vo = (torch.empty_like(x) for x in rows)
    mv.paged_kv_read(cache, table, lens, cu, ko, vo)
    assert torch.equal(ko, rows[0])                            # held exactly in every format
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(mv.paged_attention_workspace(n_seq, hq, hk, d), dtype=torch.uint8, device="cuda")
    mv.paged_attention(q, cache, table, lens, float(LN2), out, ws)

    w = torch.ones(n_seq, n, 1, 1, dtype=torch.float64, device="cuda")
    w[:, late, 0, 0] = torch.tensor([2.0 ** by for _, _, _, by in todo], dtype=torch.float64)
    w /= w.sum(1, keepdim=True)
    held = vo.double().reshape(n_seq, n, hk, d)
    ref = (w * held).sum(1).repeat_interleave(hq // hk, 1)
    mag = (w * held.abs()).sum(1).repeat_interleave(hq // hk, 1)
    tol = 2.0 ** -8 * ref.abs() + ((2.0 ** -16 if dtype == mv.DTYPE_BF16 else 2.0 ** -11) + 2.0 ** -20 + (n + 8) * 2.0 ** -23) * mag
    off = ((out.double() - ref).abs() / tol).amax((1, 2)).cpu()  # a NaN stays one
    bad = [(c, float(o)) for c, o in zip(todo, off) if not o <= 1.0]
    assert not bad, f"{len(bad)} of {n_seq}: {bad[:8]}"
