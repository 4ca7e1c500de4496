"""The operators around a paged serving step on the host (no GPU needed): refusals before anything is launched, the binding's
own checks, frequencies as parts of a turn, and the arithmetic that the kernels' comments rely on."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import paged_step

INVALID, SHAPE = 1, 2
FAKE = 0x100000                                 # never dereferenced: every call here fails its checks first


def rows(ptr=FAKE, ts=1024, hs=128):
    return mv._Rows(ptr, ts, hs)


BAD_ROWS = [dict(ptr=None), dict(ptr=FAKE + 2), dict(ts=-8), dict(ts=1028), dict(hs=132), dict(ts=64), dict(hs=64),
            dict(ts=2 ** 30)]


def resize(by=FAKE, n_seq=2, page=16, n_pages=8, table=FAKE, ld=4, pages=4, lens=FAKE, free=FAKE, cu=FAKE, pos=FAKE,
           slots=FAKE, n_rows=4):
    return mv.lib().paged_kv_resize(by, n_seq, page, n_pages, table, ld, pages, lens, free, cu, pos, slots, n_rows, None)


def test_resize_refusals():
    for kw in (dict(by=None), dict(table=None), dict(lens=None), dict(free=None), dict(cu=None), dict(cu=None, pos=None),
               dict(n_seq=-1), dict(n_rows=-1), dict(slots=FAKE + 4), dict(pos=FAKE + 2), dict(by=FAKE + 1), dict(free=FAKE + 2)):
        assert resize(**kw) == INVALID, kw
    for kw in (dict(n_seq=4097), dict(page=8), dict(page=24), dict(page=2048), dict(n_pages=0), dict(pages=0), dict(ld=3),
               dict(ld=1 << 28, pages=1 << 28)):
        assert resize(**kw) == SHAPE, kw


def rope(q=None, k=None, n=3, hq=4, hk=2, d=128, qg=FAKE, kg=FAKE, eps=1e-6, pos=FAKE, turns=FAKE, rot=128, nb=0, qo=None,
         ko=None):
    return mv.lib().qk_norm_rope(q or rows(), k or rows(), n, hq, hk, d, qg, kg, eps, pos, turns, rot, nb, qo or rows(),
                                 ko or rows(), None)


def test_rope_refusals():
    for kw in BAD_ROWS:
        for name in ("q", "k", "qo", "ko"):
            assert rope(**{name: rows(**kw)}) == INVALID, (name, kw)
    for name in ("qo", "ko"):                                 # rows that overlap may be read, not written
        assert rope(**{name: rows(ts=128, hs=128)}) == INVALID
    for kw in (dict(n=-1), dict(pos=None), dict(turns=None), dict(turns=FAKE + 4), dict(pos=FAKE + 2), dict(qg=FAKE + 8),
               dict(kg=FAKE + 2), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(nb=2)):
        assert rope(**kw) == INVALID, kw
    for kw in (dict(d=8), dict(d=72), dict(d=272, rot=0), dict(rot=8), dict(rot=144), dict(rot=-16), dict(d=64, rot=128),
               dict(hq=-1), dict(hk=257)):
        assert rope(**kw) == SHAPE, kw
    assert rope(n=0) == rope(hq=0, hk=0) == 0                 # nothing to do
    assert rope(hq=0, q=rows(ptr=None, ts=0, hs=0), qo=rows(ptr=None, ts=0, hs=0), k=rows(ptr=None)) == INVALID


def test_binding_refusals():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        mv.qk_norm_rope(t, t, None, None, 1e-6, pos, None)    # not on a GPU
    with pytest.raises(ValueError):
        mv.qk_norm_rope(None, None, None, None, 1e-6, pos, None)
    for bad in (0, 8, 24):
        with pytest.raises(ValueError):
            mv.Rope(bad, device="cpu")
    for kw in (dict(theta=0.0), dict(theta=float("inf")), dict(freqs=[1.0] * 7), dict(freqs=[float("nan")] * 8)):
        with pytest.raises(ValueError):
            mv.Rope(16, device="cpu", **kw)
    with pytest.raises(ValueError):
        mv.PagedKV.zeros(2, 16, 2, 48, dtype=mv.DTYPE_E2M1, device="cpu")
    with pytest.raises(ValueError):                           # on a CPU
        mv.PagedKV.zeros(2, 16, 2, 64, dtype=mv.DTYPE_E2M1, device="cpu")


def test_frequencies_as_parts_of_a_turn():
    for kw, freqs in ((dict(theta=10000.0), [10000.0 ** (-2 * i / 64) for i in range(32)]),
                      (dict(freqs=[0.0, -0.25, 7.5, 2 * math.pi] + [1e-12] * 28), [0.0, -0.25, 7.5, 2 * math.pi] + [1e-12] * 28)):
        r = mv.Rope(64, device="cpu", **kw)
        got = [x % 2 ** 64 for x in r.turns.tolist()]
        for g, f in zip(got, freqs):
            want = Fraction(f) / Fraction(2 * math.pi) % 1
            off = abs(Fraction(g, 2 ** 64) - want)
            assert min(off, 1 - off) <= Fraction(1, 2 ** 52) * max(1, abs(Fraction(f)))


def bf16(x):
    return torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).double().numpy()


def test_product_with_the_reciprocal_scale_rounds_as_the_quotient():
    """x / s to the nearest 4-bit value: fp32 x * (1 / s) brought to multiples of 2^-11 by adding 6144 is on the same side of
    every border as the quotient, for every scale byte and bf16 value, and on it where the quotient is."""
    borders = [Fraction(b) for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)]
    for byte in (*range(1, 24), *range(112, 136), *range(0xC8, 0xE3)):
        s = np.float32(paged_step.scale_value(byte))
        inv = np.float32(1.0) / s
        for b in borders:
            x = float(b) * float(s)
            assert float(bf16(x)) == x                        # a bf16 value is there
            near = np.array([x], dtype=np.float32).view(np.uint32)[0] + (np.arange(-2, 3).astype(np.int64) << 16)
            for v in near.astype(np.uint32).view(np.float32):
                y = np.float32(np.float32(float(v) * float(inv) + 6144.0) - np.float32(6144.0))
                q = Fraction(float(v)) / Fraction(float(s))
                assert (q > b) - (q < b) == (Fraction(float(y)) > b) - (Fraction(float(y)) < b), (byte, b, v)


def test_oracle_quantise():
    x = np.zeros((8, 32))
    x[0, 0] = 6.0                                             # scale 1
    x[0, 1:9] = [0.25, 0.26, 0.75, 1.25, -1.75, 2.5, -3.5, 5.0]
    x[1, 0] = 1e6                                             # over 6 * 10240
    x[2, 3] = 6 * 2.0 ** -18                                  # half of the least scale: to 0
    x[3, 3] = 6 * 2.0 ** -17
    x[4, 20] = np.nan
    x[5, 2] = np.inf
    x[6, 16] = 6 * 1.0625                                     # half way between scales 1 and 1.125: to 1
    x[7, 16] = -6 * 1.1875                                    # between 1.125 and 1.25: to 1.25
    code, byte = paged_step.quantise(x)
    assert byte[0, 0] == 15 << 3 and byte[0, 1] == 0
    assert code[0, :9].tolist() == [7, 0, 1, 2, 2, 8 + 4, 4, 8 + 6, 6]
    assert byte[1, 0] == paged_step.TOP_BYTE and code[1, 0] == 7
    assert byte[2, 0] == 0 and not code[2].any()
    assert byte[3, 0] == 1 and code[3, 3] == 7
    assert byte[4].tolist() == [0, 255] and byte[5].tolist() == [255, 0]
    assert byte[6, 1] == 15 << 3 and code[6, 16] == 7 and byte[7, 1] == (15 << 3) + 2 and code[7, 16] == 8 + 7
    v = paged_step.stored_value(paged_step.pack(code), byte)
    assert v[0, :9].tolist() == [6, 0, 0.5, 1, 1, -2, 2, -4, 4] and np.isnan(v[4, 16:]).all() and not np.isnan(v[4, :16]).any()
    assert np.array_equal(bf16(v[:4]), v[:4]) and np.abs(v[np.isfinite(v)]).max() <= 65504


def test_oracle_resize():
    lens, table, free = [5, 33, 0, 16], [[7, 0, 0], [2, 4, 6], [0, 0, 0], [1, 0, 0]], [2, 3, 5, 9, 9, 9, 9, 9]
    got = paged_step.resize([20, -30, 1, -16], lens, table, free, 16)
    # given up: 1 (sequence 3), then 6, 4; taken: 4 by sequence 0, 6 by sequence 2
    assert got[0] == [25, 3, 1, 0] and got[1].tolist() == [[7, 4, 0], [2, 4, 6], [6, 0, 0], [1, 0, 0]]
    assert got[2] == [3, 3, 5, 1, 6, 4, 9, 9] and got[3] == [0, 20, 20, 21, 21]
    assert got[4] == list(range(5, 25)) + [0] and got[5] == [7 * 16 + p for p in range(5, 16)] + [4 * 16 + p for p in range(9)] + [96]


def test_rope_of_no_tokens_wants_no_positions():
    assert rope(n=0, pos=None) == 0
    assert rope(n=1, pos=None) == INVALID and rope(n=0, pos=None, turns=None) == INVALID
    assert rope(n=0, pos=FAKE + 2) == INVALID


def test_product_with_the_reciprocal_scale_rounds_as_the_quotient_for_every_value():
    """The argument of the test above for all scale bytes and all bf16 values from 2^-6 to 8 scales (below, monotonic rounding
    leaves them under the first border, 0.25): products have 8 + 24 bits from 2^-37 up, so that they and their sums with 6144
    are exact in fp64 and each is rounded to fp32 once, as a fused multiply-add does."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    every = (np.arange(0x7f80, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)   # bf16 >= 0, finite, in order
    sides = 0
    for byte in range(1, paged_step.TOP_BYTE + 1):
        s = np.float32(paged_step.scale_value(byte))
        inv = float(np.float32(1.0) / s)
        x = every[(every >= float(s) / 64) & (every <= 8 * float(s))]
        y = ((x * inv + 6144.0).astype(np.float32) - np.float32(6144.0)).astype(np.float64)
        # x against border times scale, which has 7 bits: exact
        assert np.array_equal(np.sign(x[:, None] - borders * float(s)), np.sign(y[:, None] - borders)), byte
        assert y[0] < 0.25
        sides += len(x)
    assert sides > 200000
