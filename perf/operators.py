"""Measured cases of the serving operators: attention over packed prompts, writing rows into a paged key-value cache
and reading them back (bf16, or 8 bits with a power-of-two scale for each row), and attention of one new token for each
sequence over such a cache.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
framework's entry points; ``exact`` is the definition in 64 bits. Lengths follow from the case, values from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX, EXP_BIAS = -100, 120, 127


def listed():
    return [
        # one chat session of the 7B shape (32 heads of 128, every head with its own keys) after a page of text: latency
        dict(name="decode_b1_7b", op="decode", n_seq=1, max_len=1027, ragged=0, heads=32, kv_heads=32, dim=128,
             page=16, bits=16),
        # a busy server: 64 sequences of all ages, grouped heads, the cache held in 8 bits, small pages
        dict(name="decode_b64_ragged_e4m3", op="decode", n_seq=64, max_len=8191, ragged=11, heads=32, kv_heads=8,
             dim=128, page=16, bits=8),
        # sixteen long documents side by side, bf16: the largest read of a cache
        dict(name="decode_b16_long", op="decode", n_seq=16, max_len=24576, ragged=0, heads=64, kv_heads=8, dim=128,
             page=64, bits=16),
        # three sequences, one of them very long: few rows, so the length has to be split; an odd group of heads of 64
        dict(name="decode_b3_split_d64_e4m3", op="decode", n_seq=3, max_len=100003, ragged=5, heads=20, kv_heads=4,
             dim=64, page=32, bits=8),
        # one decode step's new rows (a token for each of 48 sequences) quantised into the cache and read back
        dict(name="write_step_e4m3", op="write", n_seq=48, max_len=4099, ragged=3, rows=1, heads=8, kv_heads=8,
             dim=128, page=16, bits=8),
        # the keys and values of a batch of prompts written after prefill, quantised, and read back
        dict(name="write_prompts_e4m3", op="write", n_seq=24, max_len=2500, ragged=7, rows=0, heads=8, kv_heads=8,
             dim=128, page=64, bits=8),
        # a parked bf16 cache of the small 64-wide configuration brought back into one piece
        dict(name="read_small_bf16", op="read", n_seq=2, max_len=333, ragged=2, heads=4, kv_heads=4, dim=64, page=16,
             bits=16),
        # long parked sequences in 8 bits brought back as bf16
        dict(name="read_long_e4m3", op="read", n_seq=6, max_len=30011, ragged=9, heads=8, kv_heads=8, dim=128,
             page=128, bits=8),
        # a handful of short chat turns prefilled together: latency
        dict(name="prompt_short_d64", op="prompt", n_seq=5, max_len=97, ragged=4, heads=8, kv_heads=8, dim=64),
        # a prefill batch of the 7B shape with lengths from a word to a page
        dict(name="prompt_ragged_7b", op="prompt", n_seq=12, max_len=2048, ragged=6, heads=32, kv_heads=32, dim=128),
        # one long document, grouped heads: the largest product
        dict(name="prompt_8k_gqa", op="prompt", n_seq=1, max_len=8192, ragged=0, heads=32, kv_heads=8, dim=128),
        # two odd lengths, an odd group of 64-wide heads
        dict(name="prompt_odd_d64", op="prompt", n_seq=2, max_len=4001, ragged=8, heads=14, kv_heads=2, dim=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "read", "prompt", "prompt"])
    dim = rng.choice([64, 128, 128, 32, 16]) if rng.random() < 0.3 else rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16])
    while kv_heads * group > 64:
        group = max(1, group // 2)
    case = dict(op=op, ragged=rng.randrange(1, 1000) if rng.random() < 0.8 else 0, dim=dim, kv_heads=kv_heads)
    if op == "prompt":
        most = _log(rng, 1, 6000)
        # scores of the plain form: sequences x heads x length^2 within the largest listed case's
        room = (8192 * 8192 * 32) // (most * most * kv_heads * group)
        case.update(n_seq=_log(rng, 1, max(1, min(24, room))), max_len=most, heads=kv_heads * group)
        return case
    case.update(page=rng.choice([16, 16, 32, 48, 64, 128, 256]), bits=rng.choice([8, 8, 16]))
    most = _log(rng, 1, 60000)
    while op != "decode" and kv_heads * dim * most > 100_000_000:
        most //= 2
    rows = (16 * 24576 * 8 * 128) // (kv_heads * dim * most)     # sequences that keep within the largest listed case
    if op != "decode":
        rows //= 4
    case.update(n_seq=_log(rng, 1, max(1, min(200, rows))), max_len=most,
                heads=kv_heads * group if op == "decode" else kv_heads)
    if op == "write":
        case["rows"] = rng.choice([0, 0, 1, 5])
    return case


def _lens(case):
    """Each sequence's length: all the largest, or spread over the logarithm with one the largest."""
    n, most = case["n_seq"], case["max_len"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random(case["ragged"])
    lens = [_log(r, 1, most) for _ in range(n)]
    lens[r.randrange(n)] = most
    return lens


def _rows(case, lens):
    """Rows of each sequence that a write or a read takes: all of them, or the last few."""
    k = case.get("rows", 0)
    return [min(n, k) if k else n for n in lens]


def work(case):
    lens, d, hq, hk = _lens(case), case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "prompt":
        t = sum(lens)
        return dict(bytes=2 * d * t * (2 * hq + 2 * hk), flops=2 * d * hq * sum(n * (n + 1) for n in lens))
    held = d + 1 if case["bits"] == 8 else 2 * d                  # bytes of one row of the cache
    if case["op"] == "decode":
        return dict(bytes=2 * hk * held * sum(lens) + 4 * d * hq * len(lens), flops=4 * d * hq * sum(lens))
    rows = sum(_rows(case, lens)) * hk * 2
    if case["op"] == "read":
        return dict(bytes=rows * (held + 2 * d), flops=rows * d)
    return dict(bytes=rows * (2 * d + held + 2 * d), flops=2 * rows * d)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rows_like_a_model(g, *shape):
    """Keys and values as layers give them: the rows' sizes differ, and a few columns are much larger than the rest."""
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
    x[..., 3::29] *= 3.0
    return x.to(torch.bfloat16)


def _quantise(x):
    """(e4m3, exponent byte) of each row of x in 32 bits: the smallest power of two with the row inside +-448 of it."""
    x = x.float()
    f, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(f > 0.875, e - 8, e - 9)
    e = torch.where(f == 0, torch.full_like(e, EXP_MIN), e).clamp(EXP_MIN, EXP_MAX)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + EXP_BIAS).to(torch.uint8)


def _value(x, e):
    """What stored rows stand for, in 32 bits."""
    return x.float() if e is None else torch.ldexp(x.float(), e.to(torch.int32)[..., None] - EXP_BIAS)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, d, hq, hk = _lens(case), case["dim"], case["heads"], case["kv_heads"]
    n = len(lens)
    s = dict(case=case, scale=d ** -0.5, lens=lens)
    if case["op"] == "prompt":
        t = sum(lens)
        s.update(q=_normal(g, t, hq, d), k=_normal(g, t, hk, d), v=_rows_like_a_model(g, t, hk, d))
        s["out"] = torch.empty_like(s["q"])
        s["starts"] = torch.tensor([sum(lens[:i]) for i in range(n)], device="cuda")
        s["lens_dev"] = torch.tensor(lens, device="cuda")
        if own:
            import medusa_tree_speculative_verify_gb300 as mv
            s["plan"] = mv.PromptPlan(lens, hq // hk)
        return s
    page = case["page"]
    need = [-(-x // page) for x in lens]
    pages = sum(need) + 3                                          # a few pages stay free
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    cols = torch.arange(max(need), device="cuda")[None, :]
    needed = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(needed, 0) - needed
    s["table"] = torch.where(cols < needed, order[(first + cols).clamp(max=pages - 1)],
                             torch.zeros_like(order[:1])).contiguous()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = (pages, hk, page, d)
    s["k_exp"] = s["v_exp"] = None
    if case["op"] == "write":                                      # an empty pool
        kind = torch.float8_e4m3fn if case["bits"] == 8 else torch.bfloat16
        s["k_pages"], s["v_pages"] = torch.zeros(shape, device="cuda").to(kind), torch.zeros(shape, device="cuda").to(kind)
        if case["bits"] == 8:
            s["k_exp"] = torch.zeros(shape[:-1], dtype=torch.uint8, device="cuda")
            s["v_exp"] = torch.zeros(shape[:-1], dtype=torch.uint8, device="cuda")
    else:
        s["k_pages"], s["v_pages"] = _normal(g, *shape), _rows_like_a_model(g, *shape)
        if case["bits"] == 8:
            s["k_pages"], s["k_exp"] = _quantise(s["k_pages"])
            s["v_pages"], s["v_exp"] = _quantise(s["v_pages"])
    if case["op"] == "decode":
        s["q"] = _normal(g, n, hq, d)
        s["out"] = torch.empty_like(s["q"])
    else:
        rows = _rows(case, lens)
        t = sum(rows)
        cu = [sum(rows[:i]) for i in range(n + 1)]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        if case["op"] == "write":
            s["k"], s["v"] = _rows_like_a_model(g, t, hk, d), _rows_like_a_model(g, t, hk, d)
        s["k_out"] = torch.empty(t, hk, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        import medusa_tree_speculative_verify_gb300 as mv
        s["cache"] = mv.PagedKV(k=s["k_pages"], v=s["v_pages"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        if case["op"] == "decode":
            s["ws"] = torch.zeros(mv.paged_attention_workspace(n, hq, hk, d), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import medusa_tree_speculative_verify_gb300 as mv
        if op == "prompt":
            mv.prompt_attention(s["q"], s["k"], s["v"], s["plan"], s["scale"], s["out"])
            return s["out"]
        if op == "decode":
            mv.paged_attention(s["q"], s["cache"], s["table"], s["seq_lens"], s["scale"], s["out"], s["ws"])
            return s["out"]
        if op == "write":
            mv.paged_kv_append(s["k"], s["v"], s["cu"], s["cache"], s["table"], s["seq_lens"])
        mv.paged_kv_read(s["cache"], s["table"], s["seq_lens"], s["cu"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if op == "prompt":
        return _plain_prompt(s)
    if op == "decode":
        return _plain_decode(s)
    page, slot = _places(s)
    if op == "write":
        if s["k_exp"] is None:
            s["k_pages"][page, :, slot] = s["k"]
            s["v_pages"][page, :, slot] = s["v"]
        else:
            k8, ke = _quantise(s["k"])
            v8, ve = _quantise(s["v"])
            s["k_pages"].view(torch.uint8)[page, :, slot] = k8.view(torch.uint8)
            s["v_pages"].view(torch.uint8)[page, :, slot] = v8.view(torch.uint8)
            s["k_exp"][page, :, slot] = ke
            s["v_exp"][page, :, slot] = ve
    return (_read_rows(s["k_pages"], s["k_exp"], page, slot).to(torch.bfloat16),
            _read_rows(s["v_pages"], s["v_exp"], page, slot).to(torch.bfloat16))


def _places(s):
    """Page and slot of every packed row: row i of a sequence is position len - rows + i."""
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    i = torch.arange(s["k_out"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    pos = lens[b] - cu[b + 1] + i
    page = s["case"]["page"]
    return s["table"][b, pos // page].long(), pos % page


def _read_rows(pages, exp, page, slot):
    if exp is None:
        return pages[page, :, slot].float()
    return _value(pages.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn), exp[page, :, slot])


def _read_all(pages, exp, table):
    """[sequences, kv heads, table positions, dim] of what the pages stand for, in 32 bits."""
    if exp is None:
        x = pages[table].float()
    else:
        x = _value(pages.view(torch.uint8)[table].view(torch.float8_e4m3fn), exp[table])
    b, n, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, n * p, d)


def _plain_decode(s):
    table, lens = s["table"].long(), s["seq_lens"]
    k, v = _read_all(s["k_pages"], s["k_exp"], table), _read_all(s["v_pages"], s["v_exp"], table)
    b, hk, n, d = k.shape
    q = s["q"].float().view(b, hk, -1, d)
    seen = (torch.arange(n, device="cuda")[None, :] < lens[:, None])[:, None, None, :]
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = torch.where(seen[:, 0, 0, :][:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.reshape(b, -1, d).to(torch.bfloat16)


def _plain_prompt(s):
    t, hq, d = s["q"].shape
    hk = s["k"].shape[1]
    lens, n = s["lens_dev"], s["case"]["max_len"]
    pos = torch.arange(n, device="cuda")
    real = pos[None, :] < lens[:, None]                            # [sequences, n]
    at = (s["starts"][:, None] + pos[None, :]).clamp(max=t - 1)    # a place in the pack for every padded one
    b = at.shape[0]
    q = s["q"][at].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    k = s["k"][at].float().permute(0, 2, 3, 1)[:, :, None]
    v = s["v"][at].float().permute(0, 2, 1, 3)[:, :, None]
    x = torch.matmul(q, k)
    x *= s["scale"]
    x.masked_fill_(pos[None, :] > pos[:, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[real].to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits

def _grid(x):
    """(values, exponents) of rows rounded to e4m3 under their power of two, in 64 bits: nearest, ties to even."""
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(a / E4M3_MAX))
    e = torch.where(a > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where((a > 0) & (a <= E4M3_MAX * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(a > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _softmax_product(q, k, v, scale, seen):
    """sum_j softmax_j(scale q.k_j) v_j over the seen keys; q [rows, dim], k, v [keys, dim], all in 64 bits."""
    x = (q @ k.T) * scale
    x[~seen.expand_as(x)] = -math.inf
    x = torch.exp(x - x.max(dim=-1, keepdim=True).values)
    return (x @ v) / x.sum(dim=-1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    lens, d, hq, hk = s["lens"], case["dim"], case["heads"], case["kv_heads"]
    group = hq // hk
    if case["op"] == "prompt":
        if 4 * d * hq * sum(n * n for n in lens) > 6e12:           # about ten seconds in 64 bits
            return None
        out, at = torch.zeros(sum(lens), hq, d, dtype=torch.float64, device="cuda"), 0
        for n in lens:
            seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
            for h in range(hq):
                kh = h // group
                out[at:at + n, h] = _softmax_product(s["q"][at:at + n, h].double(), s["k"][at:at + n, kh].double(),
                                                     s["v"][at:at + n, kh].double(), s["scale"], seen)
            at += n
        return out
    page = case["page"]

    def row(name, b, n):
        """Every stored row of sequence b as [positions, kv heads, dim] in 64 bits."""
        ids = s["table"][b, : -(-n // page)].long()
        x = s[name + "_pages"]
        if x.dtype == torch.bfloat16:
            x = x[ids].double()
        else:
            x = x.view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(torch.float32).double()
            x *= torch.exp2(s[name + "_exp"][ids].double() - EXP_BIAS)[..., None]
        return x.permute(0, 2, 1, 3).reshape(-1, hk, d)[:n]

    if case["op"] == "decode":
        out = torch.zeros(len(lens), hq, d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            k, v = row("k", b, n), row("v", b, n)
            seen = torch.ones(1, n, dtype=torch.bool, device="cuda")
            for h in range(hk):
                rows = slice(h * group, (h + 1) * group)
                out[b, rows] = _softmax_product(s["q"][b, rows].double(), k[:, h], v[:, h], s["scale"], seen)
        return out
    if case["op"] == "write":
        if case["bits"] == 8:
            return _grid(s["k"].double()), _grid(s["v"].double())
        return s["k"].double(), s["v"].double()
    return (torch.cat([row("k", b, n) for b, n in enumerate(lens)]),
            torch.cat([row("v", b, n) for b, n in enumerate(lens)]))
