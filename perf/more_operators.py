"""What a serving step does around the paged 8-bit key/value cache, as measured cases.

Norms of each query and key head with the rotary positions in the same pass, the
block tables and slot maps of a batch built on the GPU, attention with a sliding
window and first positions that stay visible, and attention for a batch that
shares a long prefix; each in a plain form of elementary torch operations and as
calls of the package's entry points.

The cache.  A block holds 64 positions of one head: E4M3 codes and one power of
two for the keys, and the same for the values (the byte b stands for
2^(b - 127)).  Keys lie as [dim / 16][64 positions][16 dims]; values as
[4][dim][16 positions], where position t = 32u + 16e + 8m + 4h + j of the block
has chunk 2u + h and byte 8e + 4m + j.  A table gives each sequence its blocks.
"""
import math
import random

import torch

own = False

BLOCK = 64
EPS = 1e-6

# The heads of the projections that this repository times: 7168 = 56 x 128
# attention values, QKV width 21504, 37,810 rows.
STEP_ROWS, STEP_HEADS = 37810, 56


def listed():
    return [
        # queries and keys of a video step, views of its QKV product, (time, height, width) positions
        dict(name="norm_step", op="norm", rows=STEP_ROWS, heads=STEP_HEADS, kv_heads=STEP_HEADS, dim=128, pairs="16,24,24",
             split=False, weight=True),
        # one decoded token of each of 32 sequences: latency
        dict(name="norm_token", op="norm", rows=32, heads=32, kv_heads=8, dim=128, pairs="64", split=True, weight=True),
        # one more token for each of 32 requests: latency
        dict(name="extend_token", op="extend", seqs=32, new=1, past=16383, columns=260, short=False),
        # ragged prompts of new and running requests
        dict(name="extend_prompts", op="extend", seqs=1001, new=1000, past=3001, columns=64, short=False),
        # a fourth of 32 requests is done: latency
        dict(name="release_few", op="release", seqs=32, past=16383, columns=260, keep=0),
        # a fourth of a large batch is done, whose first 5 blocks are everybody's
        dict(name="release_batch", op="release", seqs=4099, past=8000, columns=130, keep=5),
        # one token for each of 32 ragged sequences, the last 4096 positions and the first 4
        dict(name="window_token", op="window", seqs=32, new=1, past=16383, ragged=True, q_heads=32, kv_heads=8, dim=128,
             mask=1, window=4096, sinks=4),
        # causal prompts of ragged lengths through a short window
        dict(name="window_prompt", op="window", seqs=4, new=4001, past=0, ragged=True, q_heads=32, kv_heads=8, dim=128,
             mask=1, window=1000, sinks=4),
        # a chunk of a video step: runs of 256 positions see one another, a long window and the first run
        dict(name="window_step", op="window", seqs=1, new=4096, past=12345, ragged=False, q_heads=STEP_HEADS,
             kv_heads=STEP_HEADS, dim=128, mask=256, window=4096, sinks=256),
        # one token for each of 64 requests with a common prompt
        dict(name="shared_batch", op="shared", seqs=64, new=1, past=1023, ragged=True, prefix=256, q_heads=32, kv_heads=8,
             dim=128),
        # a few tokens each of a few requests, small heads
        dict(name="shared_few", op="shared", seqs=7, new=3, past=200, ragged=True, prefix=63, q_heads=16, kv_heads=2, dim=64),
        # questions of ragged lengths about one long document
        dict(name="shared_prompts", op="shared", seqs=16, new=64, past=0, ragged=True, prefix=512, q_heads=32, kv_heads=8,
             dim=128),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dim = rng.choice([64, 128])
    op = rng.choice(["norm", "extend", "release", "window", "window", "shared", "shared"])
    if op == "norm":
        # one to three axes in (near) equal shares, the rotated pairs a multiple of 8, or no rotation
        total = rng.choice([dim // 2, dim // 2, dim // 4])
        axes = rng.randint(1, 3)
        share = [total // axes] * axes
        share[0] += total - sum(share)
        heads = rng.randint(1, 56)
        return dict(op=op, rows=_log(rng, 1, 37000), heads=heads, kv_heads=rng.randint(1, heads), dim=dim,
                    pairs=",".join(map(str, share)) if rng.random() < 0.8 else "", split=rng.random() < 0.5,
                    weight=rng.random() < 0.8)
    if op == "extend":
        seqs = _log(rng, 1, 4096)
        new, past = _log(rng, 1, 900000 // seqs + 1), _log(rng, 1, 20000)
        return dict(op=op, seqs=seqs, new=new, past=past, columns=(new + past) // BLOCK + 1 + rng.randint(0, 9),
                    short=rng.random() < 0.2)
    if op == "release":
        past = _log(rng, 1, 8000)
        return dict(op=op, seqs=_log(rng, 1, 4096), past=past, columns=past // BLOCK + 1 + rng.randint(0, 9),
                    keep=rng.choice([0, 0, 1, 7]))
    kv_heads, group = rng.randint(1, 12), rng.choice([1, 2, 3, 4, 5, 8])
    tokens = rng.random() < 0.5
    if op == "window":
        case = dict(op=op, ragged=True, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, window=_log(rng, 1, 5000),
                    sinks=rng.choice([0, 1, 4, 64, 100]))
        if tokens:
            seqs = _log(rng, 1, 32)
            return dict(case, seqs=seqs, new=rng.choice([1, 1, 1, 2, 3]), past=_log(rng, 1, 200000 // seqs) - 1, mask=1)
        return dict(case, seqs=rng.randint(1, 4), new=_log(rng, 16, 3000), past=_log(rng, 1, 9000) - 1,
                    mask=rng.choice([0, 1, 1, 256]))
    case = dict(op=op, ragged=True, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if tokens:
        return dict(case, seqs=_log(rng, 1, 64), new=rng.choice([1, 1, 1, 2, 3]), past=_log(rng, 1, 1000) - 1,
                    prefix=_log(rng, 1, 400))
    return dict(case, seqs=rng.randint(1, 16), new=_log(rng, 4, 64), past=_log(rng, 1, 300) - 1, prefix=_log(rng, 1, 400))


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def _lengths(case):
    """[(new rows, positions after them)] of a case's sequences: the first is the largest.  After a shared prefix the
    positions count it."""
    r = random.Random("%(seqs)d %(new)d %(past)d" % case)
    common = BLOCK * case.get("prefix", 0)
    got = [(case["new"], common + case["past"] + case["new"])]
    for _ in range(1, case["seqs"]):
        n = r.randint(1, case["new"]) if case["ragged"] else case["new"]
        past = r.randint(0, case["past"]) if case["ragged"] else case["past"]
        got.append((n, common + past + n))
    return got


def _limit(pos, length, mask):
    return length if mask == 0 else min(length, (pos // mask + 1) * mask)


def _visible(case, pos, length):
    """(first positions, first of the others, end) that the row at pos sees."""
    end = _limit(pos, length, case.get("mask", 1))
    low = max(0, pos + 1 - case["window"]) if "window" in case else 0
    return min(case.get("sinks", 0), low), low, end


def work(case):
    op = case["op"]
    if op == "norm":
        pairs = [int(p) for p in case["pairs"].split(",") if p]
        heads = case["heads"] + case["kv_heads"]
        n = case["rows"] * heads * case["dim"]
        return {"bytes": 4 * n + case["rows"] * 4 * len(pairs), "flops": 4 * n + 6 * case["rows"] * heads * sum(pairs)}
    if op == "extend":
        # lengths and counts in and out, positions and slots, and half the blocks that the rows could take
        rows = case["seqs"] * case["new"]
        return {"bytes": 16 * case["seqs"] + 12 * rows + 4 * (rows // BLOCK), "flops": 4 * rows}
    if op == "release":
        # lengths in and out, marks, and a fourth of the blocks: entries read, and the stack
        back = max(0, case["past"] // BLOCK // 2 - case["keep"]) * case["seqs"] // 4
        return {"bytes": 12 * case["seqs"] + 8 * back, "flops": case["seqs"] + back}
    seqs, dim = _lengths(case), case["dim"]
    rows = sum(n for n, _ in seqs)
    seen = keys = 0
    for n, length in seqs:
        for i in range(n):
            first, low, end = _visible(case, length - n + i, length)
            seen += first + end - low
        first, low, _ = _visible(case, length - n, length)
        keys += first + length - low
    if op == "shared":
        keys -= (len(seqs) - 1) * BLOCK * case["prefix"]
    return {"bytes": 4 * rows * case["q_heads"] * dim + 2 * keys * case["kv_heads"] * dim,
            "flops": 4 * dim * case["q_heads"] * seen}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _keys_laid(c):
    """[n, heads, 64, dim] -> [n, heads, dim / 16, 64, 16]"""
    n, h, t, d = c.shape
    return c.reshape(n, h, t, d // 16, 16).transpose(2, 3).contiguous()


def _keys_flat(c):
    n, h, g, t, _ = c.shape
    return c.transpose(2, 3).reshape(n, h, t, g * 16)


def _values_laid(c):
    """[n, heads, 64, dim] -> [n, heads, 4, dim, 16]"""
    n, h, t, d = c.shape
    return c.reshape(n, h, 2, 2, 2, 2, 4, d).permute(0, 1, 2, 5, 7, 3, 4, 6).reshape(n, h, 4, d, 16)


def _values_flat(c):
    n, h, _, d, _ = c.shape
    return c.reshape(n, h, 2, 2, d, 2, 2, 4).permute(0, 1, 2, 5, 6, 3, 7, 4).reshape(n, h, BLOCK, d)


def _power(b):
    """2^(b - 127) of bytes 1..254, exactly."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _decode(codes, powers):
    """Codes [n, heads, 64, dim] and bytes [n, heads] -> binary32 values."""
    return codes.view(torch.float8_e4m3fn).float() * _power(powers)[..., None, None]


def _plain_norm(s):
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        f = x.float()
        f = f * torch.rsqrt((f * f).mean(dim=-1, keepdim=True) + EPS)
        if w is not None:
            f = f * w.float()
        if s["tables"]:
            cs = torch.cat([t[s["positions"][:, a].long()] for a, t in enumerate(s["tables"])], dim=1)
            c, n = cs[:, None, :, 0], cs[:, None, :, 1]
            pairs = c.shape[-1]
            turned = f[..., :2 * pairs]
            a, b = (turned[..., :pairs], turned[..., pairs:]) if s["split"] else (turned[..., 0::2], turned[..., 1::2])
            p, q = a * c - b * n, b * c + a * n
            turned = torch.cat([p, q], dim=-1) if s["split"] else torch.stack([p, q], dim=-1).flatten(-2)
            f = torch.cat([turned, f[..., 2 * pairs:]], dim=-1)
        got.append(f.to(torch.bfloat16))
    return got


def _plain_release(s):
    """Blocks of finished requests go back on the stack, in order; their lengths become 0."""
    column = torch.arange(s["table"].shape[1], device="cuda")
    blocks = (s["past"].long() + BLOCK - 1) // BLOCK
    back = (s["done"][:, None] != 0) & (column >= s["keep"]) & (column < blocks[:, None])
    freed = s["table"][back]
    count = s["free_count"].long()
    s["free"][count + torch.arange(freed.shape[0], device="cuda")] = freed
    return [torch.where(s["done"] != 0, 0, s["past"]), (count + freed.shape[0]).int(), s["free"]]


def _plain_extend(s):
    """Rows, lengths and new blocks of every request, in order; positions and slots of the rows."""
    past, rows, free_count = s["past"].long(), s["rows"], s["free_count"].long()
    ends = torch.cumsum(s["more"].long(), 0).clamp(max=rows)
    row_start = torch.cat([ends.new_zeros(1), ends])
    lens = past + row_start[1:] - row_start[:-1]
    have, need = (past + BLOCK - 1) // BLOCK, (lens + BLOCK - 1) // BLOCK
    taken = torch.cumsum(need - have, 0)
    # the j-th block taken is the j-th from the top of the stack
    column = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (column >= have[:, None]) & (column < need[:, None])
    place = free_count - 1 - ((taken - (need - have))[:, None] + column - have[:, None])
    block = torch.where(place >= 0, s["free"][place.clamp(0, s["free"].shape[0] - 1)], -1)
    s["table"].copy_(torch.where(fresh, block, s["table"]))
    # each row's sequence, position and slot; -1 for the rows that are left
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(ends, row, right=True)
    used = seq < past.shape[0]
    seq = seq.clamp(max=past.shape[0] - 1)
    pos = past[seq] + row - row_start[seq]
    page = s["table"][seq, (pos // BLOCK).clamp(max=s["table"].shape[1] - 1)].long()
    slots = torch.where(used & (page >= 0), page * BLOCK + pos % BLOCK, -1)
    positions = torch.where(used, pos, -1).int()
    left, missing = (free_count - taken[-1:]).clamp(min=0), (taken[-1:] - free_count).clamp(min=0)
    return [row_start.int(), lens.int(), left.int(), missing.int(), positions[:, None], slots, s["table"]]


def _rows_of(s):
    """Each sequence's rows padded to the largest count: row numbers, which of them are real, and positions."""
    step = torch.arange(s["new_max"], device="cuda")
    count = s["row_start"][1:] - s["row_start"][:-1]
    row = (s["row_start"][:-1, None] + step).clamp(max=s["q"].shape[0] - 1)
    return row, step < count[:, None], s["lens"][:, None] - count[:, None] + step


def _pool(s):
    """Keys and values of the pool [blocks, heads, 64, dim], binary32."""
    return (_decode(_keys_flat(s["cache"][0]), s["cache"][2]), _decode(_values_flat(s["cache"][1]), s["cache"][3]))


def _gather(x, table):
    """[sequences, heads, positions, dim] of a table's blocks."""
    n, blocks = table.shape
    return x[table.long()].transpose(1, 2).reshape(n, x.shape[1], blocks * BLOCK, x.shape[3])


def _plain_window(s):
    n, length, group = s["new_max"], s["len_max"], s["q"].shape[1] // s["cache"][0].shape[1]
    k, v = (_gather(x, s["table"])[:, :, :length] for x in _pool(s))
    seqs, heads, _, dim = k.shape
    row, real, pos = _rows_of(s)
    q = s["q"][row].float().reshape(seqs, n, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, heads, group * n, dim)
    limit = s["lens"][:, None].expand(-1, n)
    if s["mask"]:
        limit = torch.minimum(limit, (pos // s["mask"] + 1) * s["mask"])
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"]).reshape(seqs, heads, group, n, length)
    key = torch.arange(length, device="cuda")
    hidden = (key >= limit[:, :, None]) | ((key <= pos[:, :, None] - s["window"]) & (key >= s["sinks"]))
    p.masked_fill_(hidden[:, None, None], float("-inf"))
    p.sub_(p.amax(dim=-1, keepdim=True)).exp_()
    total = p.sum(dim=-1)
    o = torch.matmul(p.reshape(seqs, heads, group * n, length), v.contiguous()).reshape(seqs, heads, group, n, dim)
    o = (o / total[..., None]).permute(0, 3, 1, 2, 4).reshape(seqs, n, heads * group, dim)
    return o[real].to(torch.bfloat16)


def _plain_shared(s):
    """The rows of all sequences against the prefix, each sequence's against its own positions, one softmax."""
    blocks, group = s["shared"].shape[0], s["q"].shape[1] // s["cache"][0].shape[1]
    common = blocks * BLOCK
    pool = _pool(s)
    k0, v0 = (_gather(x, s["shared"][None])[0] for x in pool)
    heads, _, dim = k0.shape
    rows, n, seqs = s["q"].shape[0], s["new_max"], s["lens"].shape[0]
    q = s["q"].float().reshape(rows, heads, group, dim).permute(1, 0, 2, 3).reshape(heads, rows * group, dim)
    p0 = torch.matmul(q, k0.transpose(1, 2).contiguous()).mul_(s["scale"])
    top0 = p0.amax(dim=-1)
    # the sequences' own positions
    length = s["len_max"] - common
    k1, v1 = (_gather(x, s["table"][:, blocks:])[:, :, :length] for x in pool)
    row, real, pos = _rows_of(s)
    x = s["q"][row].float().reshape(seqs, n, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(seqs, heads, n * group, dim)
    p1 = torch.matmul(x, k1.transpose(2, 3).contiguous()).mul_(s["scale"])
    hidden = common + torch.arange(length, device="cuda") > pos[:, :, None]
    p1.reshape(seqs, heads, n, group, length).masked_fill_(hidden[:, None, :, None], float("-inf"))
    # one maximum and sum
    top = torch.maximum(top0.reshape(heads, rows, group)[:, row].permute(1, 0, 2, 3).reshape(seqs, heads, n * group),
                        p1.amax(dim=-1))
    p1.sub_(top[..., None]).exp_()
    own_sum, own_out = p1.sum(dim=-1), torch.matmul(p1, v1.contiguous())
    by_row = lambda t, w: t.reshape(seqs, heads, n, group, w).transpose(1, 2)[real]  # noqa: E731  [rows, heads, group, w]
    top = by_row(top, 1).squeeze(-1).permute(1, 0, 2).reshape(heads, rows * group)
    p0.sub_(top[..., None]).exp_()
    total = p0.sum(dim=-1).reshape(heads, rows, group).transpose(0, 1) + by_row(own_sum, 1).squeeze(-1)
    o = torch.matmul(p0, v0).reshape(heads, rows, group, dim).transpose(0, 1) + by_row(own_out, dim)
    return (o / total[..., None]).reshape(rows, heads * group, dim).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, *shape, sigma=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(sigma).to(torch.bfloat16)


def _ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _rope_inputs(gen, case, rows):
    """Tables of each axis (angle of position p and pair j: p 10000^(-j / pairs), formed in 64 bits) and the rows'
    positions: on one axis anywhere in a long context, on several a grid read row by row."""
    if not case["pairs"]:
        return [], None
    pairs = [int(p) for p in case["pairs"].split(",")]
    size = [131072] if len(pairs) == 1 else [97] * len(pairs)
    tables = []
    for n, p in zip(size, pairs):
        angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(p, device="cuda", dtype=torch.float64) / p)
        tables.append(torch.stack([angle.cos(), angle.sin()], dim=-1).float())
    if len(pairs) == 1:
        positions = torch.randint(0, size[0], (rows, 1), generator=gen, device="cuda", dtype=torch.int32)
    else:
        at = torch.arange(rows, device="cuda") + int(torch.randint(0, 97, (1,), generator=gen, device="cuda"))
        width = [53, 31, 97][-len(pairs):]
        cols = []
        for w in reversed(width):
            cols.append(at % w)
            at = at // w
        positions = torch.stack(cols[::-1], dim=1).to(torch.int32)
    return tables, positions


def _norm_inputs(gen, case):
    """Queries and keys as views of one QKV product, heads of several sizes, weights around one."""
    rows, heads, kv_heads, dim = case["rows"], case["heads"], case["kv_heads"], case["dim"]
    x = _normal(gen, rows, heads + 2 * kv_heads, dim)
    x *= torch.exp2(torch.randint(-3, 4, (1, heads + 2 * kv_heads, 1), generator=gen, device="cuda").float()).bfloat16()
    weight = lambda: (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).bfloat16() if case["weight"] else None  # noqa: E731
    tables, positions = _rope_inputs(gen, case, rows)
    return dict(q=x[:, :heads], k=x[:, heads:heads + kv_heads], q_weight=weight(), k_weight=weight(), tables=tables,
                positions=positions, split=case["split"])


def _table_inputs(gen, case):
    """Requests that hold blocks of a pool in use, what is free on a stack; a fourth of the requests is done.  A short
    pool cannot give all that is asked for.  The rows have room for the largest step, as in a captured graph."""
    seqs, columns, new = case["seqs"], case["columns"], case.get("new", 0)
    pick = lambda low, high: torch.randint(low, high + 1, (seqs,), generator=gen, device="cuda")  # noqa: E731
    past, more = pick(0, case["past"]), pick(min(1, new), new)
    blocks = (past + BLOCK - 1) // BLOCK
    used = int(blocks.sum())
    free = seqs * (new // BLOCK + 1)
    if case.get("short"):
        free //= 8
    order = torch.randperm(used + free, generator=gen, device="cuda").int()
    table = torch.full((seqs, columns), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(columns, device="cuda") < blocks[:, None]] = order[:used]
    stack = torch.full((free + seqs * -(-case["past"] // BLOCK),), -1, dtype=torch.int32, device="cuda")
    stack[:free] = order[used:]
    return dict(past=past.int(), more=more.int(), table=table, free=stack, free_count=_ints([free]), rows=seqs * new,
                keep=case.get("keep", 0), done=(torch.rand(seqs, generator=gen, device="cuda") < 0.25).int())


def _cache_for(gen, case, seqs):
    """A pool with a few blocks more than the sequences take, whose codes are of a key channel that stands out and of
    values of several sizes; the tables, lengths and row starts.  A shared prefix's blocks stand in every table."""
    heads, dim, common = case["kv_heads"], case["dim"], case.get("prefix", 0)
    blocks = [-(-length // BLOCK) - common for _, length in seqs]
    pool = common + sum(blocks) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").int()
    table = torch.zeros(len(seqs), common + max(blocks), dtype=torch.int32, device="cuda")
    table[:, :common] = order[:common]
    at = common
    for b, n in enumerate(blocks):
        table[b, common:common + n] = order[at:at + n]
        at += n

    def codes(x, laid):
        x = x.to(torch.bfloat16).float()
        amax = x.abs().amax(dim=(2, 3))
        bits = amax.view(torch.int32)  # the byte of the smallest power of two p with amax <= 448 p
        power = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_(min=1)
        x = (x * _power(254 - power)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return laid(x), power.to(torch.uint8)

    x = torch.randn(pool, heads, BLOCK, dim, generator=gen, device="cuda")
    x[..., 3] *= 6.0
    k, kp = codes(x, _keys_laid)
    x = torch.randn(pool, heads, BLOCK, dim, generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-2, 3, (pool, heads, 1, 1), generator=gen, device="cuda").float())
    v, vp = codes(x, _values_laid)
    starts = [0]
    for n, _ in seqs:
        starts.append(starts[-1] + n)
    return dict(cache=(k, v, kp, vp), table=table, lens=_ints([s[1] for s in seqs]), row_start=_ints(starts), rows=starts[-1],
                shared=table[0, :common].clone())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    if op == "norm":
        s = _norm_inputs(gen, case)
    elif op in ("extend", "release"):
        s = _table_inputs(gen, case)
    else:
        seqs = _lengths(case)
        s = _cache_for(gen, case, seqs)
        s.update(q=_normal(gen, s["rows"], case["q_heads"], case["dim"]), scale=case["dim"] ** -0.5, mask=case.get("mask", 1),
                 window=case.get("window", 0), sinks=case.get("sinks", 0), new_max=max(n for n, _ in seqs),
                 len_max=max(length for _, length in seqs))
    s["op"] = op
    if own:
        import nvfp4_activation_quantization_segment_amd as nv

        if op == "extend":
            s["step"] = nv.KvStep.empty(case["seqs"], s["rows"])  # kept from step to step
        elif op in ("window", "shared"):
            s["kv"] = nv.KvCache(*s["cache"])
    return s


def run(state):
    s, op = state, state["op"]
    if own:
        import nvfp4_activation_quantization_segment_amd as nv

        if op == "norm":
            return list(nv.norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], eps=EPS, tables=s["tables"],
                                     positions=s["positions"], split=s["split"]))
        if op == "extend":
            g = nv.kv_extend(s["past"], s["more"], s["table"], s["free"], s["free_count"], s["step"])
            return [g.row_start, g.lens, g.free_count, g.missing, g.positions, g.slots, s["table"]]
        if op == "release":
            lens, count = nv.kv_release(s["past"], s["done"], s["table"], s["free"], s["free_count"], keep=s["keep"])
            return [lens, count, s["free"]]
        if op == "window":
            return nv.kv_attention(s["q"], s["kv"], s["row_start"], s["lens"], s["table"], scale=s["scale"],
                                   causal_block=s["mask"], max_len=s["len_max"], window=s["window"], sinks=s["sinks"])
        return nv.kv_attention(s["q"], s["kv"], s["row_start"], s["lens"], s["table"], scale=s["scale"], causal_block=1,
                               max_len=s["len_max"], shared=s["shared"])
    return {"norm": _plain_norm, "extend": _plain_extend, "release": _plain_release, "window": _plain_window,
            "shared": _plain_shared}[op](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _exact_norm(s):
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        if w is not None:
            x = x * w.double()
        out = x.clone()
        half = sum(t.shape[1] for t in s["tables"])
        i = 0
        for a, t in enumerate(s["tables"]):
            for j in range(t.shape[1]):
                p, q = (i, i + half) if s["split"] else (2 * i, 2 * i + 1)
                turn = t.double()[s["positions"][:, a].long(), j]
                c, n = turn[:, :1], turn[:, 1:]
                out[:, :, p] = x[:, :, p] * c - x[:, :, q] * n
                out[:, :, q] = x[:, :, q] * c + x[:, :, p] * n
                i += 1
        got.append(out)
    return got


def _exact_release(s):
    past, done, table = s["past"].tolist(), s["done"].tolist(), s["table"].tolist()
    count = int(s["free_count"])
    stack, room = s["free"].tolist()[:count], s["free"].tolist()
    for b, length in enumerate(past):
        if done[b]:
            stack += table[b][s["keep"]:-(-length // BLOCK)]
            past[b] = 0
    return [_ints(past), _ints([len(stack)]), _ints(stack + room[len(stack):])]


def _exact_extend(s):
    past, more, table = s["past"].tolist(), s["more"].tolist(), s["table"].tolist()
    stack = s["free"].tolist()[:int(s["free_count"])]
    row_start, lens, positions, slots, missing = [0], [], [], [], 0
    for b, n in enumerate(more):
        n = min(n, s["rows"] - row_start[-1])
        for pos in range(past[b], past[b] + n):
            if pos % BLOCK == 0:
                missing += not stack
                table[b][pos // BLOCK] = stack.pop() if stack else -1
            page = table[b][pos // BLOCK]
            positions.append(pos)
            slots.append(page * BLOCK + pos % BLOCK if page >= 0 else -1)
        row_start.append(row_start[-1] + n)
        lens.append(past[b] + n)
    room = [-1] * (s["rows"] - len(positions))
    return [_ints(row_start), _ints(lens), _ints([len(stack)]), _ints([missing]), _ints(positions + room)[:, None],
            torch.tensor(slots + room, dtype=torch.int64, device="cuda"), _ints(table)]


def _slot(t, dim):
    """Byte offsets of position t (a tensor) in a block's keys and values, [len(t), dim]."""
    d = torch.arange(dim, device=t.device)
    t = t[:, None]
    k = (d // 16) * (BLOCK * 16) + t * 16 + d % 16
    chunk = 2 * (t // 32) + t // 4 % 2
    v = chunk * (dim * 16) + d * 16 + 8 * (t // 16 % 2) + 4 * (t // 8 % 2) + t % 4
    return k, v


def _exact_attention(s, case):
    dim, (k_codes, v_codes, k_powers, v_powers) = case["dim"], s["cache"]
    pool, heads = k_powers.shape
    codes = [c.reshape(pool, heads, BLOCK * dim) for c in (k_codes, v_codes)]
    scale = [torch.exp2(p.double() - 127.0) for p in (k_powers, v_powers)]
    out = torch.empty(s["rows"], case["q_heads"], dim, dtype=torch.float64, device="cuda")
    group, common = case["q_heads"] // heads, case.get("prefix", 0)
    for b, (n, length) in enumerate(_lengths(case)):
        pos = torch.arange(length, device="cuda")
        page = s["table"][b].long()[pos // BLOCK]
        if common:
            page[:common * BLOCK] = s["shared"].long()[pos[:common * BLOCK] // BLOCK]
        r0 = int(s["row_start"][b])
        bounds = torch.tensor([_visible(case, length - n + i, length) for i in range(n)], device="cuda")
        seen = (pos < bounds[:, 2:]) & ((pos >= bounds[:, 1:2]) | (pos < bounds[:, :1]))
        there = _slot(pos % BLOCK, dim)
        for h in range(heads):
            k, v = (codes[w][page, h].gather(1, there[w]).view(torch.float8_e4m3fn).double() * scale[w][page, h][:, None]
                    for w in range(2))
            for g in range(h * group, (h + 1) * group):
                p = s["q"][r0:r0 + n, g].double() @ k.t() * s["scale"]
                p = torch.where(seen, p, float("-inf"))
                p = torch.exp(p - p.amax(dim=-1, keepdim=True))
                out[r0:r0 + n, g] = p @ v / p.sum(dim=-1, keepdim=True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] in ("extend", "release"):
        return _exact_extend(s) if case["op"] == "extend" else _exact_release(s)
    return _exact_attention(s, case)
