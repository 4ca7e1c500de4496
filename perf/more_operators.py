"""Measured cases of the operators around a paged serving step: lengths, block tables and slot maps that follow requests as
they grow and shrink, norms of the heads of Q and K with the rotation by position, rows of a key-value cache held in 4 bits
(written and read back), and attention of one new token for each sequence over such a cache.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64) or, with ``own`` set,
through the framework's entry points; ``exact`` is the definition in 64 bits. Lengths follow from the case, values from the
seed.
"""
import math
import random

import torch

own = False

GROUP = 16                        # elements that share a scale byte
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE_MAX = 10240.0


def listed():
    return [
        # one decode step of a busy server: every sequence takes a token, all of which are then given up again
        dict(name="resize_step_b48", op="resize", n_seq=48, max_len=4099, ragged=3, page=16, grow=1),
        # a tree of 64 tokens for each of 300 sequences, none of them accepted
        dict(name="resize_tree_b300", op="resize", n_seq=300, max_len=9001, ragged=5, page=32, grow=64),
        # a queue of prompts let in at once, and cancelled
        dict(name="resize_prompts_b200", op="resize", n_seq=200, max_len=8192, ragged=8, page=16, grow=0),
        # the new token of one chat session of the 7B shape (32 heads of 128, each with its own keys): latency
        dict(name="rope_step_b1_7b", op="rope", tokens=1, heads=32, kv_heads=32, dim=128, rot=128, pairs="halves",
             fused=True, gain=True, far=1027),
        # one long document, grouped heads: the largest
        dict(name="rope_8k_gqa", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, pairs="halves",
             fused=True, gain=True, far=0),
        # an odd group of 64-wide heads of which half is turned, neighbours as pairs, far positions
        dict(name="rope_odd_d64_part", op="rope", tokens=6928, heads=14, kv_heads=2, dim=64, rot=32, pairs="neighbours",
             fused=False, gain=True, far=900001),
        # one decode step's new rows (a token for each of 48 sequences) written and read back
        dict(name="write_step_e2m1", op="write", n_seq=48, max_len=4099, ragged=3, rows=1, kv_heads=8, dim=128, page=16),
        # the keys and values of a batch of prompts written after prefill, and read back
        dict(name="write_prompts_e2m1", op="write", n_seq=24, max_len=2500, ragged=7, rows=0, kv_heads=8, dim=128,
             page=64),
        # one chat session of the 7B shape after a page of text: latency
        dict(name="decode_b1_7b_e2m1", op="decode", n_seq=1, max_len=1027, ragged=0, heads=32, kv_heads=32, dim=128,
             page=16),
        # a busy server: 64 sequences of all ages, grouped heads, small pages
        dict(name="decode_b64_ragged_e2m1", op="decode", n_seq=64, max_len=8191, ragged=11, heads=32, kv_heads=8,
             dim=128, page=16),
        # sixteen long documents side by side: the largest read of a cache
        dict(name="decode_b16_long_e2m1", op="decode", n_seq=16, max_len=24576, ragged=0, heads=64, kv_heads=8, dim=128,
             page=64),
        # three sequences, one of them very long, so the length has to be split; an odd group of heads of 64
        dict(name="decode_b3_split_d64_e2m1", op="decode", n_seq=3, max_len=100003, ragged=5, heads=20, kv_heads=4,
             dim=64, page=32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["resize", "rope", "rope", "write", "decode", "decode", "decode"])
    ragged = rng.randrange(1, 1000) if rng.random() < 0.8 else 0
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    if op == "resize":
        most = _log(rng, 1, 20000)
        n_seq = _log(rng, 1, max(1, min(4096, 400_000 // most)))
        # 0: let in whole; a few tokens or a tree for each; -1: some sequences grow, some shrink, some stay
        return dict(op=op, n_seq=n_seq, max_len=most, ragged=ragged, page=page, grow=rng.choice([0, 1, 1, 5, 64, -1]))
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16])
    while kv_heads * group > 64:
        group = max(1, group // 2)
    if op == "rope":
        dim = rng.choice([32, 64, 80, 96, 128, 128, 256])
        rows = 8192 * 40 * 128 // ((kv_heads * group + kv_heads) * dim)
        rot = dim if rng.random() < 0.6 else rng.choice([r for r in (16, 32, 64, 128) if r <= dim])
        return dict(op=op, tokens=_log(rng, 1, max(1, rows)), heads=kv_heads * group, kv_heads=kv_heads, dim=dim, rot=rot,
                    pairs=rng.choice(["halves", "halves", "neighbours"]), fused=rng.random() < 0.5,
                    gain=rng.random() < 0.8, far=rng.choice([0, 0, _log(rng, 1, 2_000_000)]))
    dim = rng.choice([64, 128, 128, 32, 96])
    most = _log(rng, 1, 60000)
    while op == "write" and kv_heads * dim * most > 25_000_000:
        most //= 2
    rows = (16 * 24576 * 8 * 128) // (kv_heads * dim * most)     # sequences that keep within the largest listed case
    if op == "write":
        rows = rows // 16
    n_seq = _log(rng, 1, max(1, min(200, rows)))
    if op == "write":
        return dict(op=op, n_seq=n_seq, max_len=most, ragged=ragged, rows=rng.choice([0, 0, 1, 5]), kv_heads=kv_heads,
                    dim=dim, page=page)
    return dict(op=op, n_seq=n_seq, max_len=most, ragged=ragged, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                page=page)


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
    """Rows of each sequence that a write takes: all of them, or the last few."""
    k = case.get("rows", 0)
    return [min(n, k) if k else n for n in lens]


def _change(case, lens):
    """(lengths before, by how much each changes) of a resize."""
    grow = case["grow"]
    if grow == 0:
        return [0] * len(lens), lens
    if grow > 0:
        return lens, [grow] * len(lens)
    r = random.Random(case["ragged"] + 17)
    by = []
    for n in lens:
        kind = r.randrange(3)
        by.append(0 if kind == 0 else _log(r, 1, 300) if kind == 1 else -r.randrange(0, n + 1))
    return lens, by


def _pages(n, page):
    return -(-n // page)


def work(case):
    if case["op"] == "rope":
        t, rows, d = case["tokens"], case["heads"] + case["kv_heads"], case["dim"]
        # sum of squares, norm, gain; two products and a sum for what is turned
        return dict(bytes=t * (4 * rows * d + 4), flops=t * rows * (4 * d + 3 * case["rot"]))
    lens = _lens(case)
    if case["op"] == "resize":                                   # there and back
        lens, by = _change(case, lens)
        rows = sum(max(x, 0) for x in by)
        moved = sum(abs(_pages(n + x, case["page"]) - _pages(n, case["page"])) for n, x in zip(lens, by))
        return dict(bytes=2 * 12 * len(lens) + 4 * len(lens) + 12 * rows + 2 * 8 * moved, flops=4 * len(lens) + 2 * rows)
    hk, d = case["kv_heads"], case["dim"]
    held = d // 2 + d // GROUP                                    # bytes of one row of the cache
    if case["op"] == "decode":
        hq = case["heads"]
        return dict(bytes=2 * hk * held * sum(lens) + 4 * d * hq * len(lens), flops=4 * d * hq * sum(lens))
    rows = sum(_rows(case, lens)) * hk * 2
    return dict(bytes=rows * (2 * d + held + 2 * d), flops=3 * rows * d)


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rows_like_a_model(g, *shape):
    """Keys and values as layers give them: the rows' sizes differ, and a few columns are much larger than the rest."""
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
    x[..., 3::29] *= 3.0
    return x.to(torch.bfloat16)


def _scale_byte(x):
    """The byte nearest to x >= 0 (32 bits), ties to even: 5 exponent and 3 fraction bits, at most 10240."""
    f, e = torch.frexp(x)                                         # x = f 2^e, f in [0.5, 1)
    e = torch.clamp(e - 1, min=-14)                               # of the binade, the least for what is below it
    n = torch.round(torch.ldexp(x, 3 - e))                        # in eighths of the binade
    byte = (e + 14) * 8 + n.to(torch.int32)                       # 16 eighths: the next binade's first
    return byte.clamp(max=0xE2).to(torch.uint8)


def _scale_value(byte):
    b = byte.to(torch.int32)
    e, m = b >> 3, (b & 7).float()
    return torch.where(e > 0, torch.ldexp(8 + m, e - 18), torch.ldexp(m, torch.full_like(e, -17)))


def _quantise(x):
    """(packed e2m1, scale bytes) of the rows of x, two elements a byte, the first in the low half."""
    x = x.float().unflatten(-1, (-1, GROUP))
    byte = _scale_byte(x.abs().amax(-1) / 6)
    s = _scale_value(byte)[..., None]
    a = x.abs()
    # borders between neighbours times the scale are exact; a tie goes to the even one of the two
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border * s) if tie_up else (a > border * s)
    code = torch.where(s > 0, code + 8 * (x < 0).to(torch.uint8), torch.zeros_like(code)).flatten(-2)
    return (code[..., 0::2] | code[..., 1::2] << 4).contiguous(), byte


def _value(packed, byte):
    """What stored rows stand for, in 32 bits."""
    code = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).long()
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=packed.device)[code]
    return (v.unflatten(-1, (-1, GROUP)) * _scale_value(byte)[..., None]).flatten(-2)


def _table(lens, page, g):
    """A block table of pages in no order for sequences of these lengths, and the pages that stay free (a few)."""
    need = [_pages(x, page) for x in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    cols = torch.arange(max(max(need), 1), device="cuda")[None, :]
    needed = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(needed, 0) - needed
    table = torch.where(cols < needed, order[(first + cols).clamp(max=pages - 1)], torch.zeros_like(order[:1]))
    return table.contiguous(), pages, order[sum(need):]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        return _prepare_rope(s, case, g)
    lens, page = _lens(case), case["page"]
    n = len(lens)
    if case["op"] == "resize":
        before, by = _change(case, lens)
        most = max(_pages(max(a, a + x), page) for a, x in zip(before, by))
        grown = sum(max(0, _pages(a + x, page) - _pages(a, page)) for a, x in zip(before, by))
        table, pages, left = _table(before, page, g)
        pages += grown
        s["table"] = torch.zeros(n, most, dtype=torch.int32, device="cuda")
        s["table"][:, :min(most, table.shape[1])] = table[:, :most]
        free = torch.cat([left, torch.arange(pages - grown, pages, dtype=torch.int32, device="cuda")])
        free = free[torch.randperm(len(free), generator=g, device="cuda")]
        s["free"] = torch.zeros(1 + pages, dtype=torch.int32, device="cuda")      # how many, then the pages
        s["free"][0] = len(free)
        s["free"][1:1 + len(free)] = free
        s["seq_lens"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["by"] = torch.tensor(by, dtype=torch.int32, device="cuda")
        s["back"] = -s["by"]
        rows = sum(max(x, 0) for x in by) + 5                     # a few rows of padding
        s["cu"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        s["positions"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
        if own:
            import medusa_tree_speculative_verify_gb300 as mv
            s["cache"] = mv.PagedKV.zeros(pages, page, 1, 32, mv.DTYPE_E2M1)
        return s
    d, hk = case["dim"], case["kv_heads"]
    s["lens"] = lens
    s["table"], pages, _ = _table(lens, page, g)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = (pages, hk, page, d)
    if case["op"] == "write":                                     # an empty pool
        rows = _rows(case, lens)
        t = sum(rows)
        s["cu"] = torch.tensor([sum(rows[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        s["k"], s["v"] = _rows_like_a_model(g, t, hk, d), _rows_like_a_model(g, t, hk, d)
        s["k_out"] = torch.empty(t, hk, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        for x in "kv":
            s[x + "_pages"] = torch.zeros(*shape[:3], d // 2, dtype=torch.uint8, device="cuda")
            s[x + "_scale"] = torch.zeros(*shape[:3], d // GROUP, dtype=torch.uint8, device="cuda")
    else:
        hq = case["heads"]
        s["scale"] = d ** -0.5
        s["k_pages"], s["k_scale"] = _quantise(_normal(g, *shape))
        s["v_pages"], s["v_scale"] = _quantise(_rows_like_a_model(g, *shape))
        s["q"] = _normal(g, n, hq, d)
        s["out"] = torch.empty_like(s["q"])
    if own:
        import medusa_tree_speculative_verify_gb300 as mv
        s["cache"] = mv.PagedKV(k=s["k_pages"], v=s["v_pages"], k_exp=s["k_scale"], v_exp=s["v_scale"])
        if case["op"] == "decode":
            s["ws"] = torch.zeros(mv.paged_attention_workspace(n, hq, hk, d), dtype=torch.uint8, device="cuda")
    return s


def _prepare_rope(s, case, g):
    t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["fused"]:                                             # slices of one projection's output, values behind them
        x = _rows_like_a_model(g, t, hq + 2 * hk, d)
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
    else:
        s["q"], s["k"] = _rows_like_a_model(g, t, hq, d), _rows_like_a_model(g, t, hk, d)
    s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.empty(t, hk, d, dtype=torch.bfloat16, device="cuda")
    s["q_gain"] = s["k_gain"] = None
    if case["gain"]:
        s["q_gain"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        s["k_gain"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    s["positions"] = (case["far"] + torch.arange(t, device="cuda")).to(torch.int32)
    s["eps"], s["theta"] = 1e-6, 10000.0
    if own:
        import medusa_tree_speculative_verify_gb300 as mv
        s["rope"] = mv.Rope(case["rot"], theta=s["theta"], neighbours=case["pairs"] == "neighbours")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import medusa_tree_speculative_verify_gb300 as mv
        if op == "rope":
            mv.qk_norm_rope(s["q"], s["k"], s["q_gain"], s["k_gain"], s["eps"], s["positions"], s["rope"], s["q_out"],
                            s["k_out"])
            return s["q_out"], s["k_out"]
        if op == "resize":
            mv.paged_kv_resize(s["by"], s["cache"], s["table"], s["seq_lens"], s["free"], s["cu"], s["positions"],
                               s["slots"])
            mv.paged_kv_resize(s["back"], s["cache"], s["table"], s["seq_lens"], s["free"])
            return s["table"], s["seq_lens"], s["free"], s["cu"], s["positions"], s["slots"]
        if op == "decode":
            mv.paged_attention(s["q"], s["cache"], s["table"], s["seq_lens"], s["scale"], s["out"], s["ws"])
            return s["out"]
        mv.paged_kv_append(s["k"], s["v"], s["cu"], s["cache"], s["table"], s["seq_lens"])
        mv.paged_kv_read(s["cache"], s["table"], s["seq_lens"], s["cu"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if op == "rope":
        return _plain_rope(s, s["q"], s["q_gain"]), _plain_rope(s, s["k"], s["k_gain"])
    if op == "resize":
        s["cu"], s["positions"], s["slots"] = _plain_resize(s, s["by"])
        _plain_resize(s, s["back"])
        return s["table"], s["seq_lens"], s["free"], s["cu"], s["positions"], s["slots"]
    if op == "decode":
        return _plain_decode(s)
    page, slot = _places(s)
    out = []
    for x in "kv":
        packed, byte = _quantise(s[x])
        s[x + "_pages"][page, :, slot] = packed
        s[x + "_scale"][page, :, slot] = byte
        out.append(_value(s[x + "_pages"][page, :, slot], s[x + "_scale"][page, :, slot]).to(torch.bfloat16))
    return tuple(out)


def _places(s):
    """Page and slot of every packed row: row i of a sequence is position len - rows + i."""
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    i = torch.arange(s["k_out"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    pos = lens[b] - cu[b + 1] + i
    page = s["case"]["page"]
    return s["table"][b, pos // page].long(), pos % page


def _plain_resize(s, by):
    """Lengths, table and free stack as after a change; cu_rows, positions and slots of the rows that came."""
    page, table, free = s["case"]["page"], s["table"], s["free"]
    lens, by = s["seq_lens"].long(), by.long()
    had, has = -(-lens // page), -(-(lens + by) // page)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    # given up: onto the stack, the last sequence's last page first
    gone = (col >= has[:, None]) & (col < had[:, None])
    count = free[0].long()
    given = table[gone].flip(0)
    stack = torch.cat([free[1:], free[:1]])                       # room for what a masked write leaves out
    at = count + torch.arange(given.numel(), device="cuda")
    stack[at] = given
    count = count + given.numel()
    # taken: off the top, the first sequence's first page first
    new = (col >= had[:, None]) & (col < has[:, None])
    nth = torch.cumsum(new.flatten(), 0).view_as(new)             # the nth page that is taken
    s["table"].copy_(torch.where(new, stack[(count - nth).clamp(min=0)], table))
    count = count - new.sum()                                     # what is popped stays in its place behind the count
    s["free"].copy_(torch.cat([count[None].to(torch.int32), stack[:-1]]))
    s["seq_lens"].copy_(lens + by)
    rows = by.clamp(min=0)
    cu = torch.cat([rows.new_zeros(1), torch.cumsum(rows, 0)])
    i = torch.arange(s["positions"].numel(), device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    real = b < by.numel()
    b = b.clamp(max=by.numel() - 1)
    pos = torch.where(real, lens[b] + i - cu[b], torch.zeros_like(i))
    slot = s["table"][b, pos // page].long() * page + pos % page
    none = torch.full_like(i, -1)
    return cu.to(torch.int32), torch.where(real, pos, none).to(torch.int32), torch.where(real, slot, none)


def _plain_rope(s, x, gain):
    case = s["case"]
    rot, halves = case["rot"], case["pairs"] == "halves"
    x = x.float()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    if gain is not None:
        x = x * gain.float()
    freq = s["theta"] ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = s["positions"].double()[:, None, None] * freq
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    y = torch.empty_like(x)
    y[..., rot:] = x[..., rot:]
    one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., one] = x[..., one] * c - x[..., two] * n
    y[..., two] = x[..., two] * c + x[..., one] * n
    return y.to(torch.bfloat16)


def _read_all(pages, scale, table):
    """[sequences, kv heads, table positions, dim] of what the pages stand for, in 32 bits."""
    x = _value(pages[table], scale[table])
    b, n, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, n * p, d)


def _plain_decode(s):
    table, lens = s["table"].long(), s["seq_lens"]
    k, v = _read_all(s["k_pages"], s["k_scale"], table), _read_all(s["v_pages"], s["v_scale"], table)
    b, hk, n, d = k.shape
    q = s["q"].float().view(b, hk, -1, d)
    seen = (torch.arange(n, device="cuda")[None, :] < lens[:, None])[:, None, None, :]
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = torch.where(seen[:, 0, 0, :][:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.reshape(b, -1, d).to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits

def _held(x):
    """What rows (64 bits) stand for once written: nearest neighbours on the two grids, by sorting."""
    x = x.unflatten(-1, (-1, GROUP))
    grid = torch.tensor([m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 29) for m in range(8)],
                        dtype=torch.float64, device=x.device)[:0xE3]
    s = _nearest(x.abs().amax(-1) / 6, grid)[..., None]
    v = _nearest(x.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.tensor(E2M1, dtype=torch.float64, device=x.device))
    return (torch.where(s > 0, v * s, torch.zeros_like(v)) * torch.sign(x)).flatten(-2)


def _nearest(x, grid):
    """The entry of the ascending grid nearest to each x, of two equally near ones the one at an even place."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    down = (below < above) | ((below == above) & (lo % 2 == 0))
    return torch.where(down, grid[lo], grid[hi])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, s["q"], s["q_gain"]), _exact_rope(s, s["k"], s["k_gain"])
    if case["op"] == "resize":
        return _exact_resize(s)
    lens, d, hk, page = s["lens"], case["dim"], case["kv_heads"], case["page"]
    if case["op"] == "write":
        return _held(s["k"].double()), _held(s["v"].double())
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device="cuda")

    def row(name, b, n):
        """Every stored row of sequence b as [positions, kv heads, dim] in 64 bits."""
        ids = s["table"][b, :_pages(n, page)].long()
        packed, byte = s[name + "_pages"][ids].long(), s[name + "_scale"][ids].long()
        x = torch.empty(*packed.shape[:-1], d, dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = value[packed % 16], value[packed // 16]
        e, m = byte // 8, (byte % 8).double()
        scale = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e.double() - 15), m / 8 * 2.0 ** -14)
        x *= scale.repeat_interleave(GROUP, -1)
        return x.permute(0, 2, 1, 3).reshape(-1, hk, d)[:n]

    group = case["heads"] // hk
    out = torch.zeros(len(lens), case["heads"], d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        k, v = row("k", b, n), row("v", b, n)
        for h in range(hk):
            rows = slice(h * group, (h + 1) * group)
            x = (s["q"][b, rows].double() @ k[:, h].T) * s["scale"]
            x = torch.exp(x - x.max(dim=-1, keepdim=True).values)
            out[b, rows] = (x @ v[:, h]) / x.sum(dim=-1, keepdim=True)
    return out


def _exact_rope(s, x, gain):
    """Each pair of a row as a complex number times e^(i position f)."""
    case = s["case"]
    rot, d = case["rot"], case["dim"]
    x = x.double()
    x = x * (x.pow(2).sum(-1, keepdim=True) / d + s["eps"]).pow(-0.5)
    if gain is not None:
        x = x * gain.double()
    k = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = torch.outer(s["positions"].double(), torch.exp(-math.log(s["theta"]) * 2 * k / rot))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    head = x[..., :rot]
    if case["pairs"] == "halves":
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag, x[..., rot:]], dim=-1)
    z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], dim=-1)


def _exact_resize(s):
    """One page after the other, on the host."""
    page = s["case"]["page"]
    table, lens = s["table"].tolist(), s["seq_lens"].tolist()
    free = s["free"].tolist()                                     # how many, then the stack

    def change(by):
        for b in reversed(range(len(by))):
            for nth in reversed(range(_pages(lens[b] + by[b], page), _pages(lens[b], page))):
                free[0] += 1
                free[free[0]] = table[b][nth]
        cu, positions, slots = [0], [], []
        for b, x in enumerate(by):
            for nth in range(_pages(lens[b], page), _pages(lens[b] + x, page)):
                table[b][nth] = free[free[0]]
                free[0] -= 1
            for p in range(lens[b], lens[b] + x):
                positions.append(p)
                slots.append(table[b][p // page] * page + p % page)
            cu.append(len(positions))
            lens[b] += x
        return cu, positions, slots

    cu, positions, slots = change(s["by"].tolist())
    change(s["back"].tolist())
    pad = [-1] * (s["positions"].numel() - len(positions))
    return tuple(torch.tensor(x) for x in (table, lens, free, cu, positions + pad, slots + pad))
