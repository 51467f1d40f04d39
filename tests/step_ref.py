"""Plain references of the operators around the cache (CPU, numpy and torch), written from the header's formulas: norms
in 64 bits, tables request by request, attention row by row."""
import numpy as np
import torch

from tests import kv_ref

BLOCK = kv_ref.BLOCK


def norm_rope(x, weight, eps, tables, positions, split):
    """x [rows, heads, dim] bf16 -> (exact, bound on the kernel's error), 64 bits.

    The bound.  A lane adds 16 squares in four sums and the lanes of a head (at most 32) in five more steps: at most
    4 + 2 + 5 roundings of the sum, two more by the mean and eps (2^-24 each), half of which the root keeps; the root's
    instruction is off by 2^-23, the two products by 2^-24 each: below 12 * 2^-24 of n.  A rotation adds two roundings
    of each product and sum.  The result is rounded once to bf16 (half a step is 2^-8 of it, or 2^-134 where it is
    subnormal)."""
    x = x.double()
    n = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        n = n * weight.double()
    y, size = n.clone(), n.abs()
    total = sum(t.shape[1] for t in tables)
    i = 0
    for a, t in enumerate(tables):
        for j in range(t.shape[1]):
            c, s = (t[positions[:, a].long(), j, w].double()[:, None] for w in (0, 1))
            p, q = (i, i + total) if split else (2 * i, 2 * i + 1)
            y[:, :, p] = n[:, :, p] * c - n[:, :, q] * s
            y[:, :, q] = n[:, :, q] * c + n[:, :, p] * s
            size[:, :, p] = (n[:, :, p] * c).abs() + (n[:, :, q] * s).abs()
            size[:, :, q] = (n[:, :, q] * c).abs() + (n[:, :, p] * s).abs()
            i += 1
    before = 14 * 2.0 ** -24 * size
    return y, before + 2.0 ** -8 * (y.abs() + before) + 2.0 ** -134


def extend(past, more, table, stack, rows):
    """Lists -> dict of what kv_extend writes.  `table` and `stack` are changed."""
    row_start, lens, positions, slots, missing = [0], [], [], [], 0
    columns = len(table[0])
    for b, want in enumerate(more):
        n = max(0, min(want, rows - row_start[-1], 2**31 - 1 - max(past[b], 0)))
        for pos in range(past[b], past[b] + n):
            at = pos // BLOCK
            slot = -1
            if 0 <= at < columns:
                if pos % BLOCK == 0:
                    missing += not stack
                    table[b][at] = stack.pop() if stack else -1
                if table[b][at] >= 0:
                    slot = table[b][at] * BLOCK + pos % BLOCK
            positions.append(pos)
            slots.append(slot)
        row_start.append(row_start[-1] + n)
        lens.append(past[b] + n)
    room = [-1] * (rows - len(positions))
    return dict(row_start=row_start, lens=lens, positions=positions + room, slots=slots + room, free=len(stack),
                missing=missing)


def release(lens, done, table, stack, keep, capacity):
    """Lists -> lengths after it.  `stack` is changed."""
    for b in range(len(lens)):
        if done[b]:
            blocks = min(max(0, -(-lens[b] // BLOCK)), len(table[b]))
            stack += [p for p in table[b][keep:blocks] if p >= 0]
    del stack[capacity:]
    return [0 if d else n for n, d in zip(lens, done)]


def visible(pos, length, causal, window, sinks, columns=None):
    """Which of `length` keys the row at position pos sees."""
    j = np.arange(length)
    return (j < kv_ref.limit(pos, length, causal)) & ((j < sinks) | (j > pos - window) if window else True)


def attention(q, cache, row_start, lens, table, scale, c, window=0, sinks=0, shared=None):
    """out [M, heads, dim] in 64 bits (NaN in rows of no sequence), and the largest error that the kernel's own roundings
    allow each element: kv_ref.attention's bound, over the keys that a row sees.  But through a window or over a prefix
    the rounded p are summed, so that with p' = p (1 + d), |d| <= 2^-8, the quotient is off by sum p d (v - o) / sum p',
    at most 2^-8 / (1 - 2^-8) of sum p |v - o| / sum p <= a + |o|: 1.01 * 2^-8 |o| more than with the exact sum."""
    M, Hq, D = q.shape
    G = Hq // cache.heads
    out = np.full((M, Hq, D), np.nan)
    tol = np.zeros((M, Hq, D))
    common = 0 if shared is None else len(shared) * BLOCK
    for b in range(len(lens)):
        n, length = row_start[b + 1] - row_start[b], int(lens[b])
        if n <= 0 or length < 0 or length > table.shape[1] * BLOCK or (common and length - n < common):
            continue
        blocks = np.array(table[b])
        if shared is not None:
            blocks[:len(shared)] = shared
        seen = np.stack([visible(length - n + i, length, c, window, sinks) for i in range(n)])
        rows = slice(row_start[b], row_start[b] + n)
        for g in range(Hq):
            k = cache.sequence(0, g // G, blocks, length)
            v = cache.sequence(1, g // G, blocks, length)
            x = q[rows, g]
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.where(seen, x @ np.where(np.isnan(k), 0, k).T * scale, -np.inf)
                poison = (seen[:, :, None] & np.isnan(v)[None]).any(1) | (seen & np.isnan(k).any(1)[None]).any(1)[:, None]
                k, v = np.nan_to_num(k), np.nan_to_num(v)
                top = s.max(1, keepdims=True) if length else np.full((n, 1), -np.inf)
                p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                l = p.sum(1, keepdims=True)
                l = np.where(l == 0, 1.0, l)
                o, a = p @ v / l, p @ np.abs(v) / l
                ds = scale * (2.0 ** -21 * np.abs(x).max(1, keepdims=True) * (np.abs(k).sum(1).max() if length else 0) +
                              1.25 * 2 * D * 2.0 ** -24 * (np.abs(x) @ np.abs(k).T).max(1, keepdims=True, initial=0))
                ds = ds + 4 * 2.0 ** -24 * (2 * np.abs(np.where(seen, s, 0)).max(1, keepdims=True, initial=0) + 16) + \
                    (length + 64) * 2.0 ** -24
            out[rows, g] = np.where(poison, np.nan, o)
            before = (1.01 * 2.0 ** -8 + 2 * ds) * a + 1.01 * 2.0 ** -8 * np.abs(o)
            tol[rows, g] = before + 2.0 ** -8 * (np.abs(o) + before) + 1e-38
    return out, tol
