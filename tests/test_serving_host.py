"""The serving operators on the host (no GPU needed): the prompt plan's work items, the refusals of every entry point
before anything is launched, and the oracle's e4m3 against torch's type."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import medusa_tree_speculative_verify_gb300 as mv
from oracle import serving

INVALID, SHAPE, CAPACITY, CUDA = 1, 2, 4, 5
FAKE = 0x100000                                 # never dereferenced: every call here fails its checks first


@pytest.mark.parametrize("lens,group", [([1], 1), ([128], 1), ([129], 1), ([0, 5, 0, 300], 3), ([257, 1, 64], 2),
                                        ([1000, 3, 513], 8), ([], 4), ([0, 0], 1)])
def test_plan_covers_every_sub_tile_once_longest_first(lens, group):
    plan = mv.PromptPlan(lens, group)
    items = plan.items()
    assert plan.n_tokens == sum(lens) and plan.n_items == len(items)
    starts = np.cumsum([0] + lens)[:-1]
    want = {(int(s), t) for s, n in zip(starts, lens) for t in range(-(-n // 128) * group)}
    got = []
    for start, n, t, keys in items.tolist():
        assert n in [m for s, m in zip(starts, lens) if s == start and m]
        tiles = -(-n // 128) * group
        assert t % 2 == 0 and 0 <= t < tiles and keys == min(t + 1, tiles - 1) // group + 1
        got += [(start, u) for u in (t, t + 1) if u < tiles]
    assert len(got) == len(set(got)) and set(got) == want
    assert (np.diff(items[:, 3]) <= 0).all()


@pytest.mark.parametrize("lens,group,status", [([-1], 1, INVALID), ([1], 0, INVALID), ([1], 257, SHAPE),
                                               ([2 ** 31 - 1], 1, SHAPE), ([2 ** 30, 2 ** 30], 1, SHAPE),
                                               ([2 ** 29] * 3, 256, SHAPE)])
def test_plan_refusals(lens, group, status):
    arr, out = (ctypes.c_int32 * len(lens))(*lens), ctypes.c_void_p(1)
    assert mv.lib().mv_prompt_plan_create(arr, len(lens), group, ctypes.byref(out)) == status
    assert not out.value
    assert mv.lib().mv_prompt_plan_create(None, 1, 1, ctypes.byref(out)) == INVALID
    assert mv.lib().mv_prompt_plan_create(arr, 1, 1, None) == INVALID
    with pytest.raises(ValueError):
        mv.PromptPlan([-1])


# A CUDA runtime of one device whose copies from pageable memory are under way when cudaMemcpy returns, as the real one's
# may be, and come only with a synchronisation of the stream they are on.
FAKE_RUNTIME = r"""
#include <stdlib.h>
#include <string.h>
static struct { void *dst, *staged; size_t n; } late[64];
static int n_late;
int fake_late(void) { return n_late; }
static int land(void) {
  while (n_late) { --n_late; memcpy(late[n_late].dst, late[n_late].staged, late[n_late].n); free(late[n_late].staged); }
  return 0;
}
int cudaGetDeviceCount(int* n) { *n = 1; return 0; }
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaSetDevice(int d) { return d != 0; }
int cudaGetLastError(void) { return 0; }
int cudaMalloc(void** p, size_t n) { *p = calloc(n ? n : 1, 1); return 0; }
int cudaFree(void* p) { land(); free(p); return 0; }
int cudaMemcpy(void* dst, const void* src, size_t n, int kind) {
  (void)kind;
  late[n_late].staged = memcpy(malloc(n), src, n);
  late[n_late].dst = dst;
  late[n_late++].n = n;
  return 0;
}
int cudaStreamSynchronize(void* s) { return s == (void*)0 || s == (void*)1 ? land() : 0; }
int cudaDeviceSynchronize(void) { return land(); }
"""


def in_fake_runtime(tmp_path, code):
    """Runs ``code`` in a process whose library calls the runtime above; ``late()`` counts the copies not there yet."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("needs a C compiler")
    mv.lib()                                                  # built before the process starts
    src, so = tmp_path / "fake.c", tmp_path / "fake.so"
    src.write_text(FAKE_RUNTIME)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    head = "import ctypes, medusa_tree_speculative_verify_gb300 as mv\nlate = ctypes.CDLL(None).fake_late\n"
    env = dict(os.environ, LD_PRELOAD=str(so), PYTHONPATH=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    return subprocess.run([sys.executable, "-c", head + code], env=env, capture_output=True, text=True, timeout=120)


def test_plan_is_on_the_device_when_it_is_handed_out(tmp_path):
    """A first call may come on any stream, so nothing of a new plan may still be on its way."""
    r = in_fake_runtime(tmp_path, "p = mv.PromptPlan([300, 5, 900], 2)\nassert p.n_items > 0\nprint(late())")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["0"]


def test_tree_is_on_the_device_when_it_is_handed_out(tmp_path):
    r = in_fake_runtime(tmp_path, "t = mv.Tree([(0,), (1,), (0, 0)], 2)\nassert t.n_nodes == 4\nprint(late())")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["0"]


def rows(ptr=FAKE, ts=1024, hs=128):
    return mv._Rows(ptr, ts, hs)


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, dtype=mv.DTYPE_E4M3, n_pages=8, page_size=16, n_kv_heads=2,
             head_dim=128)
    d.update(kw)
    return mv._PagedKVDesc(*(d[n] for n, _ in mv._PagedKVDesc._fields_))


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_exp=None), INVALID), (dict(v_exp=None), INVALID),
              (dict(dtype=mv.DTYPE_F32), INVALID), (dict(dtype=7), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v_exp=FAKE + 4), INVALID),
              (dict(n_pages=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE),
              (dict(page_size=2048), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=257), SHAPE),
              (dict(head_dim=8), SHAPE), (dict(head_dim=72), SHAPE), (dict(head_dim=144), SHAPE)]
BAD_ROWS = [dict(ptr=None), dict(ptr=FAKE + 2), dict(ts=-8), dict(ts=1028), dict(hs=132), dict(ts=64), dict(hs=64),
            dict(ts=2 ** 30)]


def append(c=None, k=None, v=None, n=4, cu=FAKE, table=FAKE, ld=4, pages=4, lens=FAKE, n_seq=2):
    return mv.lib().paged_kv_append(k or rows(), v or rows(), n, cu, c or cache(), table, ld, pages, lens, n_seq, None)


def read(c=None, k=None, v=None, n=4, cu=FAKE, table=FAKE, ld=4, pages=4, lens=FAKE, n_seq=2):
    return mv.lib().paged_kv_read(c or cache(), table, ld, pages, lens, n_seq, cu, n, k or rows(), v or rows(), None)


def attention(c=None, q=None, out=None, heads=4, table=FAKE, ld=4, pages=4, lens=FAKE, n_seq=2, scale=0.1, ws=FAKE,
              nbytes=1 << 30):
    return mv.lib().paged_attention(q or rows(), heads, c or cache(), table, ld, pages, lens, n_seq, scale,
                                    out or rows(), ws, nbytes, None)


@pytest.mark.parametrize("call", [append, read, attention])
def test_paged_refusals_of_every_call(call):
    for kw, status in BAD_CACHES:
        assert call(cache(**kw)) == status, kw
    assert call(table=None) == call(lens=None) == INVALID
    assert call(n_seq=-1) == INVALID
    assert call(n_seq=4097) == SHAPE
    assert call(pages=0) == SHAPE and call(ld=3) == SHAPE
    assert call(ld=1 << 28, pages=1 << 28) == SHAPE           # more positions than 31 bits count
    assert call(n_seq=0) == 0                                 # nothing to do


@pytest.mark.parametrize("call", [append, read])
def test_paged_row_refusals(call):
    for kw in BAD_ROWS:
        assert call(k=rows(**kw)) == INVALID and call(v=rows(**kw)) == INVALID, kw
    assert call(cu=None) == INVALID and call(n=-1) == INVALID
    assert call(n=0) == 0
    if call is read:                                          # rows that overlap may be read, not written
        assert call(k=rows(ts=128, hs=128)) == INVALID


def test_paged_attention_refusals():
    for kw in BAD_ROWS:
        assert attention(q=rows(**kw)) == INVALID and attention(out=rows(**kw)) == INVALID, kw
    assert attention(out=rows(ts=128, hs=128)) == INVALID
    assert attention(heads=3) == attention(heads=0) == attention(heads=258) == SHAPE
    assert attention(ws=None) == attention(ws=FAKE + 4) == INVALID
    assert attention(nbytes=64) == CAPACITY
    for s in (float("nan"), float("inf"), -0.5):
        assert attention(scale=s) == INVALID
    assert mv.paged_attention_workspace(4, 8, 2, 64) > 0
    for bad in ((4097, 8, 2, 64), (4, 7, 2, 64), (4, 8, 0, 64), (4, 8, 2, 72), (4, 512, 2, 64)):
        with pytest.raises(mv.MVError):
            mv.paged_attention_workspace(*bad)


def test_prompt_attention_refusals():
    plan = mv.PromptPlan([3, 200], 2)

    def call(q=None, k=None, v=None, out=None, hq=4, hk=2, d=128, p=plan.handle, scale=0.1):
        return mv.lib().prompt_attention(q or rows(), k or rows(), v or rows(), hq, hk, d, p, scale, out or rows(), None)

    for kw in BAD_ROWS:
        for name in ("q", "k", "v", "out"):
            assert call(**{name: rows(**kw)}) == INVALID, (name, kw)
    assert call(out=rows(ts=128, hs=128)) == INVALID
    assert call(p=None) == INVALID
    assert call(hq=6) == call(hk=1) == call(hq=0, hk=0) == call(hq=512, hk=256) == SHAPE
    assert call(d=4) == call(d=136) == call(d=100) == SHAPE
    for s in (float("nan"), float("inf"), -0.5):
        assert call(scale=s) == INVALID
    if not torch.cuda.is_available():
        assert call() == CUDA                                 # a plan without a device cannot run
    empty = mv.PromptPlan([0, 0], 2)
    assert call(p=empty.handle) == 0


def test_paged_attention_of_more_positions_than_places():
    """256 units of 2^30 positions and more in one sequence: no launch could count them."""
    c = cache(n_kv_heads=256, page_size=1024, dtype=mv.DTYPE_BF16)
    assert attention(c, heads=256, q=rows(ts=1 << 20), out=rows(ts=1 << 20), ld=1 << 21, pages=(1 << 21) - 2, n_seq=1) == SHAPE


def test_scale_over_what_fp32_holds_as_a_power_of_two():
    """Scores are exponents of two in fp32: log2(e) times a scale of 3e38 is none any more."""
    plan = mv.PromptPlan([3, 200], 2)
    assert attention(scale=3e38) == INVALID
    assert mv.lib().prompt_attention(rows(), rows(), rows(), 4, 2, 128, plan.handle, 3e38, rows(), None) == INVALID


def test_binding_refuses_what_the_library_cannot_see():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mv.prompt_attention(t, t, t, mv.PromptPlan([4]), 1.0, t)   # not on a GPU
    with pytest.raises(ValueError):
        mv.PagedKV(t, t)
    with pytest.raises(ValueError):
        mv.PagedKV(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    with pytest.raises(ValueError):
        mv.PagedKV.zeros(2, 16, 2, 64, dtype=mv.DTYPE_F32, device="cpu")


def test_oracle_e4m3_is_torchs():
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(serving.e4m3_value(b.numpy()), want, equal_nan=True)
    x = np.random.default_rng(0).uniform(-448, 448, 20000) * 2.0 ** -np.random.default_rng(1).integers(0, 18, 20000)
    mid = (want[:126] + want[1:127]) / 2                      # ties
    x = np.concatenate([x, mid, -mid, [0.0, 448.0, -448.0]]).astype(np.float32)
    got = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(serving.e4m3_byte(x), got)


def test_oracle_row_exponent():
    for a, e in [(448.0, 0), (449.0, 1), (1.75, -8), (1.7578125, -7), (0.0, -100), (1e-38, -100), (3.3e38, 120),
                 (float("inf"), 120), (224.0, -1), (224.1, 0)]:
        assert serving.row_exponent([[a, 0.0, -a / 2, float("nan")]])[0] == e, a
