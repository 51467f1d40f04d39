"""Plain references of the rotary, cache and attention operators (CPU, numpy and torch), written from the header's
formulas: positions are handled one by one, block layouts through their index formulas, attention in 64 bits."""
import numpy as np
import torch

BLOCK = 64


def rotate(x, tables, positions, split, dtype=torch.float32):
    """x [rows, heads, dim] -> rotated, in `dtype` (not rounded to bf16)."""
    x = x.to(dtype)
    out = x.clone()
    total = sum(t.shape[1] for t in tables)
    i = 0
    for a, t in enumerate(tables):
        for j in range(t.shape[1]):
            c, s = (t[positions[:, a].long(), j, w].to(dtype)[:, None] for w in (0, 1))
            p, q = (i, i + total) if split else (2 * i, 2 * i + 1)
            out[:, :, p] = x[:, :, p] * c - x[:, :, q] * s
            out[:, :, q] = x[:, :, q] * c + x[:, :, p] * s
            i += 1
    return out


def key_offset(t, d):
    return (d // 16) * (BLOCK * 16) + t * 16 + d % 16


def value_offset(t, d, D):
    u, e, m, h, j = t // 32, t // 16 % 2, t // 8 % 2, t // 4 % 2, t % 4
    return (2 * u + h) * (D * 16) + d * 16 + 8 * e + 4 * m + j


def offsets(D):
    """(keys, values): byte of [position, dim] in a block of one head."""
    t, d = np.arange(BLOCK)[:, None], np.arange(D)[None, :]
    return key_offset(t, d), value_offset(t, d, D)


def e4m3_table():
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    return v.numpy()


E4M3 = e4m3_table()


def nearest_code(x):
    """The E4M3 code nearest to each x (|x| <= 448; ties to the even code, sign kept, NaN code for what is not finite)."""
    x = np.asarray(x, np.float64)
    mag = E4M3[:0x7F]  # codes 0..0x7E, increasing
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(mag, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - mag[lo], mag[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def power_for(values):
    """The power byte of one head's values in a block."""
    v = np.abs(values[np.isfinite(values)])
    amax = v.max() if v.size else 0.0
    b = 1
    while amax > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


class Cache:
    """A pool as numpy bytes; kind 0 keys, 1 values."""

    def __init__(self, blocks, heads, dim):
        self.blocks, self.heads, self.dim = blocks, heads, dim
        self.codes = [np.zeros((blocks, heads, BLOCK * dim), np.uint8) for _ in range(2)]
        self.powers = [np.ones((blocks, heads), np.uint8) for _ in range(2)]
        self.off = offsets(dim)

    def values(self, kind, page, head):
        """[64, dim] in 64 bits."""
        c = self.codes[kind][page, head][self.off[kind]]
        return E4M3[c] * 2.0 ** (int(self.powers[kind][page, head]) - 127)

    def write(self, rows, row_start, lens, table):
        """rows: (k, v) as float64 arrays [M, heads, dim]."""
        for b in range(len(lens)):
            n, length = row_start[b + 1] - row_start[b], int(lens[b])
            if n <= 0 or length < 0 or length > table.shape[1] * BLOCK:
                continue
            first = length - n
            for at in range(max(first, 0) // BLOCK, -(-length // BLOCK)):
                page = int(table[b, at])
                if page < 0 or page >= self.blocks:
                    continue
                lo, hi = max(first, at * BLOCK), min(length, (at + 1) * BLOCK)
                r0 = row_start[b] + lo - first
                for kind in range(2):
                    for h in range(self.heads):
                        x = rows[kind][r0:r0 + hi - lo, h]
                        p = power_for(x)
                        off, codes = self.off[kind], self.codes[kind][page, h]
                        if lo > at * BLOCK:
                            had = int(self.powers[kind][page, h])
                            p = max(p, had)
                            if p > had:
                                kept = off[:lo - at * BLOCK]
                                old = codes[kept]
                                again = nearest_code(E4M3[old] * 2.0 ** (had - p))
                                codes[kept] = np.where((old & 0x7F) == 0x7F, old, again)
                        if kind == 1 and power_for(x) >= 247:  # what an earlier use left may not be finite
                            codes[off[hi - at * BLOCK:]] = 0
                        most = 240.0 if p >= 247 else 448.0
                        y = np.where(np.isfinite(x), np.clip(x * 2.0 ** (127 - p), -most, most), x)
                        codes[off[lo - at * BLOCK:hi - at * BLOCK]] = nearest_code(y)
                        self.powers[kind][page, h] = p

    def sequence(self, kind, head, table_row, length):
        """The first `length` positions' values, 64 bits; NaN where the block does not exist."""
        got = np.zeros((length, self.dim))
        for at in range(-(-length // BLOCK)):
            hi = min(length, (at + 1) * BLOCK)
            page = int(table_row[at])
            if 0 <= page < self.blocks:
                got[at * BLOCK:hi] = self.values(kind, page, head)[:hi - at * BLOCK]
            else:
                got[at * BLOCK:hi] = np.nan
        return got


def limit(pos, length, c):
    return length if c == 0 else max(0, min(length, (pos // c + 1) * c))


def attention(q, cache, row_start, lens, table, scale, c, bounds=False):
    """out [M, heads, dim] in 64 bits (NaN in rows of no sequence), and with bounds=True the largest error that the
    kernel's own roundings allow each element.

    The bound: p is rounded to bf16 and the output is (half a step, 2^-8 relative, each).  A score is off by the
    query's split (2^-21 of the row's largest element, times sum |k|) and by binary32 sums of its two halves' products
    (2 dim terms, 2^-24 each, of sum |q||k|, which the halves can exceed by 2^-3); scaling and subtracting the
    reference add 4 steps of the largest score, exp2 and the sums of p and of the output the rest.  A score's error
    enters p relatively, once above and once below the fraction."""
    M, Hq, D = q.shape
    G = Hq // cache.heads
    out = np.full((M, Hq, D), np.nan)
    tol = np.zeros((M, Hq, D))
    for b in range(len(lens)):
        n, length = row_start[b + 1] - row_start[b], int(lens[b])
        if n <= 0:
            continue
        if length < 0 or length > table.shape[1] * BLOCK:
            continue  # NaN
        for g in range(Hq):
            k = cache.sequence(0, g // G, table[b], length)
            v = cache.sequence(1, g // G, table[b], length)
            for i in range(n):
                r = row_start[b] + i
                lim = limit(length - n + i, length, c)
                if lim == 0:
                    out[r, g] = 0.0
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = k[:lim] @ q[r, g] * scale
                    p = np.exp(s - s.max())
                    o = p @ v[:lim] / p.sum()
                    out[r, g] = o
                    if bounds:
                        a = p @ np.abs(v[:lim]) / p.sum()
                        ds = scale * (2.0 ** -21 * np.abs(q[r, g]).max() * np.abs(k[:lim]).sum(1) +
                                      1.25 * 2 * D * 2.0 ** -24 * (np.abs(k[:lim]) @ np.abs(q[r, g])))
                        ds = ds.max() + 4 * 2.0 ** -24 * (2 * np.abs(s).max() + 16) + (lim + 64) * 2.0 ** -24
                        tol[r, g] = (2.0 ** -8 + 2 * ds) * a + 2.0 ** -8 * (np.abs(o) + (2.0 ** -8 + 2 * ds) * a) + 1e-38
    return (out, tol) if bounds else out


def attention_fast(q, cache, row_start, lens, table, scale, c):
    """`attention` without the row loop (no bounds), for larger shapes."""
    M, Hq, D = q.shape
    G = Hq // cache.heads
    out = np.full((M, Hq, D), np.nan)
    tol = np.zeros((M, Hq, D))
    for b in range(len(lens)):
        n, length = row_start[b + 1] - row_start[b], int(lens[b])
        if n <= 0:
            continue
        lims = np.array([limit(length - n + i, length, c) for i in range(n)])
        for g in range(Hq):
            k = cache.sequence(0, g // G, table[b], length)
            v = cache.sequence(1, g // G, table[b], length)
            x = q[row_start[b]:row_start[b] + n, g]
            s = x @ k.T * scale
            hidden = np.arange(length)[None, :] >= lims[:, None]
            s = np.where(hidden, -np.inf, s)
            top = s.max(1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            l = p.sum(1, keepdims=True)
            l = np.where(l == 0, 1.0, l)
            o, a = p @ v / l, p @ np.abs(v) / l
            ds = scale * (2.0 ** -21 * np.abs(x).max(1, keepdims=True) * np.abs(k).sum(1).max() +
                          1.25 * 2 * D * 2.0 ** -24 * (np.abs(x) @ np.abs(k).T).max(1, keepdims=True))
            ds = ds + 4 * 2.0 ** -24 * (2 * np.abs(np.where(hidden, 0, s)).max(1, keepdims=True) + 16) + \
                (length + 64) * 2.0 ** -24
            rows = slice(row_start[b], row_start[b] + n)
            out[rows, g] = o
            tol[rows, g] = (2.0 ** -8 + 2 * ds) * a + 2.0 ** -8 * (np.abs(o) + (2.0 ** -8 + 2 * ds) * a) + 1e-38
    return out, tol


# Calls whose long writer and reader take several heads to a workgroup, the last of them fewer: heads, dim,
# [(past, new)] and the heads that a workgroup takes, written and read.
HEAD_LOOPS = [
    (53, 128, [(37, 5000), (0, 4000)], 3, 2),
    (57, 64, [(1, 63), (100, 8900), (0, 37)], 4, 2),
    (41, 64, [(0, 20000), (17, 10001)], 9, 2),
    (37, 64, [(63, 60001)], 16, 2),
    (35, 128, [(5, 60002)], 16, 2),
]

# Attention calls with key/value heads in multiples of 8 that take 128-row tiles with a bound of 0 or 2^20 on the
# lengths: dim, heads, query heads per key/value head, causal block, [(past, new)]; so many rows of no sequence before
# the first and after the last.
WIDE_HEADS = [
    (128, 8, 1, 1, [(0, 300), (77, 130), (0, 0), (500, 65)]), (64, 8, 3, 1, [(10, 200), (0, 129)]),
    (64, 8, 2, 1, [(30, 190), (0, 70)]), (64, 16, 1, 0, [(64, 257)]), (128, 16, 2, 100, [(0, 140), (200, 70)]),
    (64, 24, 1, 1, [(0, 100), (0, 400), (3, 90)]),
]
WIDE_LEAD = 3
