"""What lies between the QKV projection and the attention output's quantizer, as measured cases.

Rotary positions with several axes, the paged 8-bit key/value cache (written as
it is quantised, read back) and attention over it, each in a plain form of
elementary torch operations and as calls of the package's entry points.

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
MAX_CODE = 448.0  # largest E4M3 value

# The heads of the projections that this repository times: 7168 = 56 x 128
# attention values, QKV width 21504, 37,810 rows.
STEP_ROWS, STEP_HEADS, STEP_DIM = 37810, 56, 128


def listed():
    return [
        # the query third of a video step's QKV product, (time, height, width) positions
        dict(name="rope_step", op="rope", rows=STEP_ROWS, heads=STEP_HEADS, kv_heads=STEP_HEADS,
             dim=128, pairs="16,24,24", split=False),
        # image tokens, two axes, small heads, an odd row count
        dict(name="rope_image", op="rope", rows=4095, heads=24, kv_heads=24, dim=64, pairs="16,16", split=True),
        # 16 decoded tokens, half of each head rotated
        dict(name="rope_token", op="rope", rows=16, heads=32, kv_heads=8, dim=128, pairs="32", split=True),
        # the whole step's keys and values into an empty cache, keys rotated on the way
        dict(name="write_step", op="write", seqs=1, new=STEP_ROWS, past=0, ragged=False, q_heads=STEP_HEADS, heads=STEP_HEADS,
             dim=128, pairs="16,24,24", split=False),
        # ragged chunks appended to sequences of odd lengths
        dict(name="write_append", op="write", seqs=7, new=1500, past=777, ragged=True, q_heads=32, heads=8, dim=128,
             pairs="", split=False),
        # one token for each of 32 sequences
        dict(name="write_token", op="write", seqs=32, new=1, past=4095, ragged=True, q_heads=32, heads=8, dim=128,
             pairs="64", split=True),
        # a step's cache read back whole
        dict(name="read_step", op="read", seqs=1, new=STEP_ROWS, past=0, ragged=False, heads=STEP_HEADS, dim=128),
        # the newest positions of ragged sequences
        dict(name="read_ragged", op="read", seqs=5, new=700, past=900, ragged=True, heads=16, dim=64),
        # one token over a short context: latency
        dict(name="attention_token", op="attention", seqs=1, new=1, past=516, ragged=False, q_heads=32, kv_heads=8,
             dim=128, mask=1),
        # one token for each of 32 ragged sequences
        dict(name="attention_batch", op="attention", seqs=32, new=1, past=16383, ragged=True, q_heads=32, kv_heads=8,
             dim=128, mask=1),
        # causal prompts of ragged lengths
        dict(name="attention_prompt", op="attention", seqs=4, new=4001, past=0, ragged=True, q_heads=32, kv_heads=8,
             dim=128, mask=1),
        # a chunk of a video step over the whole step's cache, no mask
        dict(name="attention_step", op="attention", seqs=1, new=4096, past=STEP_ROWS - 4096, ragged=False,
             q_heads=STEP_HEADS, kv_heads=STEP_HEADS, dim=128, mask=0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dim = rng.choice([64, 128])
    # one to three axes in (near) equal shares, the rotated pairs a multiple of 8
    total = rng.choice([dim // 2, dim // 2, dim // 4])
    axes = rng.randint(1, 3)
    share = [total // axes] * axes
    share[0] += total - sum(share)
    pairs, split = ",".join(map(str, share)), rng.random() < 0.5
    op = rng.choice(["rope", "write", "read", "attention", "attention"])
    if op == "rope":
        heads = rng.randint(1, 56)
        return dict(op=op, rows=_log(rng, 1, 37000), heads=heads, kv_heads=rng.randint(1, heads), dim=dim, pairs=pairs,
                    split=split)
    if op in ("write", "read"):
        seqs, heads = _log(rng, 1, 32), rng.randint(1, 16)
        case = dict(op=op, seqs=seqs, new=_log(rng, 1, 40000 // seqs), past=_log(rng, 1, 20000 // seqs) - 1, ragged=True,
                    heads=heads, dim=dim)
        if op == "read":
            return case
        return dict(case, q_heads=heads * rng.choice([1, 2, 4]), pairs=pairs if rng.random() < 0.6 else "", split=split)
    kv_heads, group = rng.randint(1, 12), rng.choice([1, 2, 3, 4, 5, 8])
    if rng.random() < 0.5:  # tokens
        seqs = _log(rng, 1, 32)
        return dict(op=op, seqs=seqs, new=rng.choice([1, 1, 1, 2, 3]), past=_log(rng, 1, 200000 // seqs) - 1, ragged=True,
                    q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, mask=1)
    seqs = rng.randint(1, 4)
    return dict(op=op, seqs=seqs, new=_log(rng, 16, 3000), past=_log(rng, 1, 9000) - 1, ragged=True,
                q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, mask=rng.choice([0, 1, 1, 256]))


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def _lengths(case):
    """[(new rows, positions after them)] of a case's sequences: the first is the largest."""
    r = random.Random("%(seqs)d %(new)d %(past)d" % case)
    got = [(case["new"], case["past"] + case["new"])]
    for _ in range(1, case["seqs"]):
        n = r.randint(1, case["new"]) if case["ragged"] else case["new"]
        past = r.randint(0, case["past"]) if case["ragged"] else case["past"]
        got.append((n, past + n))
    return got


def _limit(pos, length, mask):
    return length if mask == 0 else min(length, (pos // mask + 1) * mask)


def work(case):
    op, dim = case["op"], case["dim"]
    if op == "rope":
        pairs = [int(p) for p in case["pairs"].split(",")]
        n = case["rows"] * case["heads"] * dim
        return {"bytes": 4 * n + case["rows"] * 4 * len(pairs), "flops": 6 * case["rows"] * case["heads"] * sum(pairs)}
    seqs = _lengths(case)
    if op == "write":
        n = sum(s[0] for s in seqs) * case["heads"] * dim
        return {"bytes": 2 * (2 * n + n), "flops": 2 * 2 * n}
    if op == "read":
        n = sum(s[0] for s in seqs) * case["heads"] * dim
        return {"bytes": 2 * (n + 2 * n), "flops": 2 * n}
    rows = sum(s[0] for s in seqs)
    keys = sum(s[1] for s in seqs)
    seen = sum(_limit(length - n + i, length, case["mask"]) for n, length in seqs for i in range(n))
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


def _power_for(amax):
    """The byte of the smallest power of two p with amax <= 448 p."""
    bits = amax.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_(min=1)


def _encode(x, powers):
    """Binary32 values [n, heads, 64, dim] -> codes, each the nearest E4M3 of x / p."""
    inverse = _power(254 - powers)[..., None, None]
    return (x * inverse).to(torch.float8_e4m3fn).view(torch.uint8)


def _finite_max(x):
    return torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=(2, 3))


def _angles(tables, positions):
    """cos and sin [rows, 1, pairs] of each row's positions."""
    cs = torch.cat([t[positions[:, a].long()] for a, t in enumerate(tables)], dim=1)
    return cs[:, None, :, 0], cs[:, None, :, 1]


def _rotate(x, tables, positions, split):
    """x [rows, heads, dim] bf16 -> the rotated heads, bf16."""
    c, s = _angles(tables, positions)
    pairs = c.shape[-1]
    f = x.float()
    turned = f[..., :2 * pairs]
    a, b = (turned[..., :pairs], turned[..., pairs:]) if split else (turned[..., 0::2], turned[..., 1::2])
    p, q = a * c - b * s, b * c + a * s
    turned = torch.cat([p, q], dim=-1) if split else torch.stack([p, q], dim=-1).flatten(-2)
    return torch.cat([turned, f[..., 2 * pairs:]], dim=-1).to(torch.bfloat16)


def _plain_write(s):
    k = _rotate(s["k"], s["tables"], s["positions"], s["split"]) if s["tables"] else s["k"]
    # the touched blocks of each sequence: positions [unit, 64], the rows that
    # land there, and what was there before
    first = s["lens"].long() - (s["row_start"][1:] - s["row_start"][:-1]).long()
    at = (first // BLOCK)[:, None] + torch.arange(s["touched"], device=first.device)
    unit = (at * BLOCK < s["lens"][:, None]).nonzero(as_tuple=True)
    at, seq = at[unit], unit[0]
    page = s["table"][seq, at].long()
    pos = at[:, None] * BLOCK + torch.arange(BLOCK, device=first.device)
    new = (pos >= first[seq][:, None]) & (pos < s["lens"][seq][:, None])
    old = pos < first[seq][:, None]
    row = (s["row_start"][seq][:, None] + pos - first[seq][:, None]).clamp(0, s["k"].shape[0] - 1)
    for x, codes, powers, laid, flat in ((k, s["cache"][0], s["cache"][2], _keys_laid, _keys_flat),
                                         (s["v"], s["cache"][1], s["cache"][3], _values_laid, _values_flat)):
        fresh = x[row].float().transpose(1, 2)  # [unit, heads, 64, dim]
        keep = new[:, None, :, None]
        fresh = torch.where(keep, fresh, torch.zeros_like(fresh))
        before = flat(codes[page])
        had = torch.where(old.any(1)[:, None], powers[page].int(), 0)
        power = torch.maximum(_power_for(_finite_max(fresh)), had)
        shrink = torch.where(had > 0, _power((127 + had - power).clamp(min=0)), 1.0)
        stored = before.view(torch.float8_e4m3fn).float() * shrink[..., None, None]
        stored = stored.to(torch.float8_e4m3fn).view(torch.uint8)
        got = torch.where(keep, _encode(fresh, power), torch.where(old[:, None, :, None], stored, before))
        codes[page] = laid(got)
        powers[page] = power.to(torch.uint8)
    return _cache_values(s["cache"])


def _cache_values(cache):
    """The cache as the numbers it holds: codes as E4M3, powers as their exponents' bytes."""
    return [cache[0].view(torch.float8_e4m3fn), cache[1].view(torch.float8_e4m3fn), cache[2], cache[3]]


def _places(s):
    """Of each output row: its sequence and position."""
    row = torch.arange(s["rows"], device=s["lens"].device)
    seq = torch.searchsorted(s["row_start"][1:].contiguous(), row.int(), right=True)
    return seq, s["lens"][seq].long() - s["row_start"][seq + 1].long() + row


def _plain_read(s):
    seq, pos = _places(s)
    page, t = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    u, e, m, h, j = t // 32, t // 16 % 2, t // 8 % 2, t // 4 % 2, t % 4
    k = s["cache"][0][page, :, :, t].flatten(-2)                      # [rows, heads, dim]
    v = s["cache"][1][page, :, 2 * u + h, :, 8 * e + 4 * m + j]
    return [(c.view(torch.float8_e4m3fn).float() * _power(p[page])[..., None]).to(torch.bfloat16)
            for c, p in ((k, s["cache"][2]), (v, s["cache"][3]))]


def _plain_attention(s):
    n, length, group = s["new_max"], s["len_max"], s["q"].shape[1] // s["cache"][0].shape[1]
    table = s["table"].long()
    seqs, dim = table.shape[0], s["q"].shape[2]
    heads = s["cache"][0].shape[1]
    k = _decode(_keys_flat(s["cache"][0]), s["cache"][2])[table]      # [seqs, blocks, heads, 64, dim]
    v = _decode(_values_flat(s["cache"][1]), s["cache"][3])[table]
    k, v = (x.transpose(1, 2).reshape(seqs, heads, -1, dim)[:, :, :length] for x in (k, v))
    step = torch.arange(n, device=table.device)
    count = s["row_start"][1:] - s["row_start"][:-1]
    row = (s["row_start"][:-1, None] + step).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().reshape(seqs, n, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, heads, group * n, dim)
    pos = s["lens"][:, None] - count[:, None] + step
    limit = s["lens"][:, None].expand(-1, n)
    if s["mask"]:
        limit = torch.minimum(limit, (pos // s["mask"] + 1) * s["mask"])
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    p = p.reshape(seqs, heads, group, n, length)
    hidden = torch.arange(length, device=table.device) >= limit[:, None, None, :, None]
    p.masked_fill_(hidden, float("-inf"))
    p.sub_(p.amax(dim=-1, keepdim=True)).exp_()
    total = p.sum(dim=-1)
    o = torch.matmul(p.reshape(seqs, heads, group * n, length), v.contiguous()).reshape(seqs, heads, group, n, dim)
    o = (o / total[..., None]).permute(0, 3, 1, 2, 4).reshape(seqs, n, heads * group, dim)
    return o[step < count[:, None]].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, *shape, sigma=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(sigma).to(torch.bfloat16)


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


def _heads_of_qkv(gen, rows, q_heads, kv_heads, dim, which):
    """The asked parts of one [rows, (q_heads + 2 kv_heads) dim] product, as views of it."""
    x = _normal(gen, rows, q_heads + 2 * kv_heads, dim)
    parts = {"q": x[:, :q_heads], "k": x[:, q_heads:q_heads + kv_heads], "v": x[:, q_heads + kv_heads:]}
    return [parts[w] for w in which]


def _cache_for(gen, seqs, heads, dim, filled):
    """A cache with a few blocks more than the sequences' tables take, the tables, lengths and row starts.  Every block
    holds codes (of a key channel that stands out and of values of several sizes), as in a pool that has been in use."""
    blocks = [-(-length // BLOCK) for _, length in seqs]
    pool = sum(blocks) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").int()
    table = torch.zeros(len(seqs), max(blocks), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    if filled:
        x = torch.randn(pool, heads, BLOCK, dim, generator=gen, device="cuda")
        x[..., 3] *= 6.0
        x = x.to(torch.bfloat16).float()
        power = _power_for(_finite_max(x))
        k, kp = _keys_laid(_encode(x, power)), power.to(torch.uint8)
        x = torch.randn(pool, heads, BLOCK, dim, generator=gen, device="cuda")
        x *= torch.exp2(torch.randint(-2, 3, (pool, heads, 1, 1), generator=gen, device="cuda").float())
        x = x.to(torch.bfloat16).float()
        power = _power_for(_finite_max(x))
        v, vp = _values_laid(_encode(x, power)), power.to(torch.uint8)
    else:
        k = torch.zeros(pool, heads, dim // 16, BLOCK, 16, dtype=torch.uint8, device="cuda")
        v = torch.zeros(pool, heads, 4, dim, 16, dtype=torch.uint8, device="cuda")
        kp, vp = (torch.ones(pool, heads, dtype=torch.uint8, device="cuda") for _ in range(2))
    starts = [0]
    for n, _ in seqs:
        starts.append(starts[-1] + n)
    to = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(cache=(k, v, kp, vp), table=table, lens=to([s[1] for s in seqs]), row_start=to(starts), rows=starts[-1])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dim = case["op"], case["dim"]
    if op == "rope":
        # the queries are a strided part of the QKV product
        x, = _heads_of_qkv(gen, case["rows"], case["heads"], case["kv_heads"], dim, "q")
        tables, positions = _rope_inputs(gen, case, case["rows"])
        return dict(op=op, x=x, tables=tables, positions=positions, split=case["split"])
    seqs = _lengths(case)
    if op == "write":
        s = _cache_for(gen, seqs, case["heads"], dim, filled=case["past"] > 0)
        k, v = _heads_of_qkv(gen, s["rows"], case["q_heads"], case["heads"], dim, "kv")
        tables, positions = _rope_inputs(gen, case, s["rows"])
        touched = max((length - 1) // BLOCK - (length - n) // BLOCK + 1 for n, length in seqs)
        return dict(s, op=op, k=k, v=v, tables=tables, positions=positions, split=case["split"], touched=touched)
    if op == "read":
        return dict(_cache_for(gen, seqs, case["heads"], dim, filled=True), op=op)
    s = _cache_for(gen, seqs, case["kv_heads"], dim, filled=True)
    q = _normal(gen, s["rows"], case["q_heads"], dim)
    return dict(s, op=op, q=q, mask=case["mask"], scale=dim ** -0.5, new_max=max(n for n, _ in seqs),
                len_max=max(length for _, length in seqs))


def run(state):
    s, op = state, state["op"]
    if own:
        import nvfp4_activation_quantization_segment_amd as nv

        if op == "rope":
            return nv.rope(s["x"], s["tables"], s["positions"], split=s["split"])
        cache = nv.KvCache(*s["cache"])
        if op == "write":
            nv.kv_write(cache, s["k"], s["v"], s["row_start"], s["lens"], s["table"], tables=s["tables"],
                        positions=s["positions"], split=s["split"])
            return _cache_values(s["cache"])
        if op == "read":
            return list(nv.kv_read(cache, s["rows"], s["row_start"], s["lens"], s["table"]))
        return nv.kv_attention(s["q"], cache, s["row_start"], s["lens"], s["table"], scale=s["scale"],
                               causal_block=s["mask"], max_len=s["len_max"])
    if op == "rope":
        return _rotate(s["x"], s["tables"], s["positions"], s["split"])
    return {"write": _plain_write, "read": _plain_read, "attention": _plain_attention}[op](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _exact_rotate(x, tables, positions, split):
    x = x.double()
    out = x.clone()
    half = sum(t.shape[1] for t in tables)
    i = 0
    for a, t in enumerate(tables):
        for j in range(t.shape[1]):
            p, q = (i, i + half) if split else (2 * i, 2 * i + 1)
            turn = t.double()[positions[:, a].long(), j]
            c, s = turn[:, :1], turn[:, 1:]
            out[:, :, p] = x[:, :, p] * c - x[:, :, q] * s
            out[:, :, q] = x[:, :, q] * c + x[:, :, p] * s
            i += 1
    return out


def _nearest_e4m3(x):
    """The nearest E4M3 value (even on ties) of |x| <= 448, in 64 bits."""
    _, e = torch.frexp(x)
    grain = torch.exp2((e.double() - 1).clamp(min=-6.0) - 3)
    return torch.round(x / grain) * grain


def _slot(t, dim):
    """Byte offsets of position t (a tensor) in a block's keys and values, [len(t), dim]."""
    d = torch.arange(dim, device=t.device)
    t = t[:, None]
    k = (d // 16) * (BLOCK * 16) + t * 16 + d % 16
    chunk = 2 * (t // 32) + t // 4 % 2
    v = chunk * (dim * 16) + d * 16 + 8 * (t // 16 % 2) + 4 * (t // 8 % 2) + t % 4
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    op, dim = case["op"], case["dim"]
    if op == "rope":
        return _exact_rotate(s["x"], s["tables"], s["positions"], s["split"])
    seqs = _lengths(case)
    k_codes, v_codes, k_powers, v_powers = s["cache"]
    pool, heads = k_powers.shape
    codes = [c.reshape(pool, heads, BLOCK * dim).view(torch.float8_e4m3fn) for c in (k_codes, v_codes)]
    scale = [torch.exp2(p.double() - 127.0) for p in (k_powers, v_powers)]
    if op == "write":
        k = _exact_rotate(s["k"], s["tables"], s["positions"], s["split"]).to(torch.bfloat16) if s["tables"] else s["k"]
        values = [c.double() for c in codes]
        powers = [p.long() for p in (k_powers, v_powers)]
        for b, (n, length) in enumerate(seqs):
            r0, first = int(s["row_start"][b]), length - n
            for at in range(first // BLOCK, -(-length // BLOCK)):
                page = int(s["table"][b, at])
                lo, hi = max(first, at * BLOCK), min(length, (at + 1) * BLOCK)
                for w, x in enumerate((k, s["v"])):
                    x = x[r0 + lo - first:r0 + hi - first].double()      # [positions, heads, dim]
                    amax = x.abs().amax(dim=(0, 2))
                    power = torch.ceil(torch.log2(amax / MAX_CODE)).long() + 127
                    power = torch.where(torch.exp2(power.double() - 128) * MAX_CODE >= amax, power - 1, power).clamp(min=1)
                    before = torch.arange(0, lo - at * BLOCK, device=x.device)
                    if len(before):
                        power = torch.maximum(power, powers[w][page])
                        there = _slot(before, dim)[w].flatten()
                        stored = values[w][page][:, there] * torch.exp2((powers[w][page] - power).double())[:, None]
                        values[w][page][:, there] = _nearest_e4m3(stored)
                    there = _slot(torch.arange(lo - at * BLOCK, hi - at * BLOCK, device=x.device), dim)[w]
                    code = _nearest_e4m3(x * torch.exp2(127.0 - power.double())[:, None])
                    values[w][page][:, there.flatten()] = code.permute(1, 0, 2).flatten(1)
                    powers[w][page] = power
        return [v.reshape(c.shape) for v, c in zip(values, (k_codes, v_codes))] + [None, None]
    if op == "read":
        got = [torch.empty(s["rows"], heads, dim, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, (n, length) in enumerate(seqs):
            pos = torch.arange(length - n, length, device="cuda")
            page = s["table"][b].long()[pos // BLOCK]
            for w in range(2):
                there = _slot(pos % BLOCK, dim)[w]
                r0 = int(s["row_start"][b])
                block = codes[w].view(torch.uint8)[page].gather(2, there[:, None].expand(-1, heads, -1))
                got[w][r0:r0 + n] = block.view(torch.float8_e4m3fn).double() * scale[w][page][..., None]
        return got
    out = torch.empty(s["rows"], case["q_heads"], dim, dtype=torch.float64, device="cuda")
    group = case["q_heads"] // heads
    for b, (n, length) in enumerate(seqs):
        pos = torch.arange(length, device="cuda")
        page = s["table"][b].long()[pos // BLOCK]
        r0 = int(s["row_start"][b])
        limit = torch.tensor([_limit(length - n + i, length, case["mask"]) for i in range(n)], device="cuda")
        there = _slot(pos % BLOCK, dim)
        for h in range(heads):
            k, v = (codes[w].view(torch.uint8)[page, h].gather(1, there[w]).view(torch.float8_e4m3fn).double() *
                    scale[w][page, h][:, None] for w in range(2))
            for g in range(h * group, (h + 1) * group):
                p = s["q"][r0:r0 + n, g].double() @ k.t() * s["scale"]
                p.masked_fill_(pos >= limit[:, None], float("-inf"))
                out[r0:r0 + n, g] = torch.softmax(p, dim=-1) @ v
    return out
