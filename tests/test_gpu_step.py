"""The operators around the cache (norms of heads, tables of a step, attention through a window and over a shared
prefix) against plain references (tests/step_ref.py)."""
import random

import numpy as np
import pytest
import torch

from tests import kv_ref, step_ref
from tests.gpu_util import device
from tests.test_gpu_attention import gen, i32, normal, same, strided, tables_for

pytestmark = pytest.mark.gpu
BLOCK = 64


@pytest.fixture(scope="module")
def nv():
    import nvfp4_activation_quantization_segment_amd as m

    device()
    return m


# ---------------------------------------------------------------------------
# norms of heads
# ---------------------------------------------------------------------------
def check_norm(got, x, weight, eps, tables, positions, split):
    want, tol = step_ref.norm_rope(x, weight, eps, tables, positions, split)
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), (err / tol).argmax())


@pytest.mark.parametrize("rows,heads,kv_heads,dim,pairs,split,layout", [
    (1, 1, 1, 16, [8], False, "plain"),
    (1, 1, 0, 32, [], False, "plain"),
    (3, 2, 1, 64, [32], True, "qkv"),
    (5, 3, 3, 64, [8, 8, 16], False, "qkv"),
    (67, 56, 7, 128, [22, 21, 21], True, "heads"),
    (129, 56, 56, 128, [16, 24, 24], False, "qkv"),
    (33, 33, 5, 128, [1, 1, 1, 13], False, "heads"),
    (19, 5, 1, 80, [40], False, "plain"),       # five units on eight lanes
    (300, 1, 2, 96, [24, 16], True, "qkv"),
    (9, 3, 2, 48, [8], True, "plain"),
    (2, 2, 5, 256, [64], True, "plain"),
    (7, 2, 1, 272, [100, 28], False, "plain"),  # 17 units on 32 lanes
    (2, 2, 2, 512, [100, 100], False, "plain"),
    (3, 300, 17, 64, [], True, "plain"),
    (8195, 24, 3, 64, [8, 12, 12], False, "qkv"),
    (8192, 5, 20, 128, [24], True, "qkv"),
])
def test_norm_rope_is_the_formula(nv, rows, heads, kv_heads, dim, pairs, split, layout):
    g = gen(rows * dim + heads)
    xs = [normal(g, rows, n, dim) * torch.exp2(torch.randint(-9, 9, (rows, n, 1), generator=g).float()).bfloat16()
          for n in (heads, kv_heads) if n]
    ws = [normal(g, dim) + 1, None if rows % 2 == 0 else normal(g, dim)]
    size = [11 + 3 * a for a in range(len(pairs))]
    tables = tables_for(pairs, size)
    positions = torch.stack([torch.randint(0, n, (rows,), generator=g) for n in size], 1).int() if pairs else None
    eps = [1e-6, 1e-3, 1.0][rows % 3]
    on = [strided(x, layout) for x in xs]
    kw = dict(eps=eps, tables=[t.cuda() for t in tables], positions=None if positions is None else positions.cuda(), split=split)
    args = dict(q_weight=ws[0].cuda()) | (dict(k=on[1], k_weight=None if ws[1] is None else ws[1].cuda()) if kv_heads else {})
    got = nv.norm_rope(on[0], **args, **kw)
    got = list(got) if kv_heads else [got]
    for y, x, w in zip(got, xs, ws):
        check_norm(y, x, w, eps, tables, positions, split)
    # into outputs of another layout, and in place, the same bytes
    outs = [strided(torch.zeros_like(x), layout) for x in xs]
    back = nv.norm_rope(on[0], **args, **kw, q_out=outs[0], **(dict(k_out=outs[1]) if kv_heads else {}))
    assert (back[0] if kv_heads else back) is outs[0]
    assert all(same(a, b) for a, b in zip(outs, got))
    nv.norm_rope(on[0], **args, **kw, q_out=on[0], **(dict(k_out=on[1]) if kv_heads else {}))
    assert all(same(a, b) for a, b in zip(on, got))
    if layout == "qkv":  # what lies beside the heads is untouched
        for x in on:
            n = x.shape[1]
            wide = torch.as_strided(x, (rows, 3 * n, dim), (3 * n * dim, dim, 1), 0)
            assert bool((wide[:, :n] == 7).all()) and bool((wide[:, 2 * n:] == 7).all())


@pytest.mark.parametrize("dim", [16, 80, 128, 512])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-6, 1.0])
def test_norms_of_large_and_small_heads(nv, dim, eps):
    """Heads whose squares leave binary32 on either side, zeros, and such heads beside ordinary ones."""
    sizes = [0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -80, 2.0 ** -62, 1.0, 2.0 ** 58, 2.0 ** 63, 2.0 ** 64, 2.0 ** 100, 3.0e38]
    x = torch.zeros(5, len(sizes), dim, dtype=torch.bfloat16)
    shape = torch.rand(5, 1, dim, generator=gen(dim)) * 2 - 1
    for i, s in enumerate(sizes):
        x[:, i] = (shape[:, 0].double() * s).to(torch.bfloat16)
    x[1, :, 1:] = 0            # one element only
    x[2, 3:, ::2] = 1.0        # and mixed with ordinary ones
    check_norm(nv.norm_rope(x.cuda(), eps=eps), x, None, eps, [], None, False)


def test_norms_of_what_is_not_finite(nv):
    """As the formula has it: an infinite element makes the others 0 and itself NaN, a NaN all of them; other heads are
    not touched by it.  A position outside its table gives NaN in the pairs it turns."""
    x = normal(gen(3), 4, 6, 128)
    x[0, 1, 7], x[1, 2, 0], x[1, 3, 127] = float("inf"), float("-inf"), float("nan")
    clean = torch.ones(4, 6, dtype=torch.bool)
    clean[0, 1] = clean[1, 2] = clean[1, 3] = False
    got = nv.norm_rope(x.cuda()).cpu()
    want, tol = step_ref.norm_rope(x, None, 1e-6, [], None, False)
    assert bool(((got.double() - want).abs() <= tol)[clean].all())
    assert bool(got[0, 1, 7].isnan()) and bool(got[1, 2, 0].isnan()) and bool(got[1, 3].isnan().all())
    assert float(got[0, 1].nan_to_num(0).abs().max()) == 0 and float(got[1, 2].nan_to_num(0).abs().max()) == 0
    tables = [t.cuda() for t in tables_for([16, 16], [5, 7])]
    positions = torch.tensor([[0, 6], [5, 0], [0, -1], [2**31 - 1, -2**31]], dtype=torch.int32)
    x = normal(gen(4), 4, 2, 128)
    for split in (False, True):
        q, k = nv.norm_rope(x.cuda(), x.cuda(), tables=tables, positions=positions.cuda(), split=split)
        assert same(q, k)
        by_axis = torch.full((128,), 2)
        for i in range(32):
            a, b = (i, i + 32) if split else (2 * i, 2 * i + 1)
            by_axis[a] = by_axis[b] = i // 16
        bad = torch.tensor([[False, False, False], [True, False, False], [False, True, False], [True, True, False]])
        assert torch.equal(q.cpu().isnan(), bad[:, by_axis][:, None, :].expand(-1, 2, -1))


def test_norm_rope_of_no_rows(nv):
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    q, k = nv.norm_rope(x, x)
    assert q.shape == k.shape == x.shape


# ---------------------------------------------------------------------------
# tables of a step
# ---------------------------------------------------------------------------
def make_requests(seed, count, past_most, new_most, columns, free_blocks, idle=0.2, capacity=None):
    """Running requests with distinct blocks and a stack: lists (past, more, table, stack)."""
    r = random.Random(seed)
    past = [r.randint(0, past_most) for _ in range(count)]
    more = [0 if r.random() < idle else r.randint(1, new_most) for _ in range(count)]
    held = [min(-(-p // BLOCK), columns) for p in past]
    order = list(range(sum(held) + free_blocks))
    r.shuffle(order)
    table, at = [], 0
    for n in held:
        table.append(order[at:at + n] + [-7] * (columns - n))
        at += n
    return past, more, table, order[at:]


def run_extend(nv, past, more, table, stack, rows, capacity=None, in_place=False, stride=None):
    capacity = capacity or len(stack) + 1
    n, columns = len(past), len(table[0])
    wide = torch.full((n, stride or columns), -9, dtype=torch.int32)
    wide[:, :columns] = torch.tensor(table, dtype=torch.int32)
    wide = wide.cuda()
    t = wide[:, :columns]
    free = i32(stack + [-5] * (capacity - len(stack)))
    count, p = i32([len(stack)]), i32(past)
    step = nv.KvStep.empty(n, rows)
    if in_place:
        step.lens, step.free_count = p, count
    got = nv.kv_extend(p, i32(more), t, free, count, step)
    assert got is step
    if not in_place:
        assert p.tolist() == past and int(count) == len(stack)
    assert free.tolist() == stack + [-5] * (capacity - len(stack))
    if stride:
        assert bool((wide[:, columns:] == -9).all())
    return step, t


def check_extend(step, t, want, table):
    assert step.row_start.tolist() == want["row_start"] and step.lens.tolist() == want["lens"]
    assert step.free_count.tolist() == [want["free"]] and step.missing.tolist() == [want["missing"]]
    assert step.positions.flatten().tolist() == want["positions"]
    assert step.slots.tolist() == want["slots"]
    assert t.tolist() == table


EXTENDS = [  # requests, past at most, new at most, columns, free blocks, rows
    (1, 0, 1, 1, 1, 1), (1, 63, 1, 2, 1, 1), (1, 64, 1, 2, 1, 1), (2, 200, 70, 6, 9, 140), (7, 500, 1, 9, 7, 7),
    (63, 300, 3, 6, 70, 100), (64, 300, 3, 6, 70, 150), (65, 300, 1, 6, 70, 65), (200, 900, 40, 16, 300, 4096),
    (200, 900, 40, 16, 300, 4097), (1023, 100, 2, 3, 2000, 2046), (1024, 100, 2, 3, 2000, 2049), (1025, 100, 9, 3, 2000, 9000),
    (3000, 1000, 1, 17, 3000, 3000), (5, 100, 5000, 90, 500, 30000), (4100, 70, 13, 3, 5000, 60000),
    (3, 0, 100000, 1700, 5000, 300000),
]


@pytest.mark.parametrize("case", range(len(EXTENDS)))
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_is_the_definition(nv, case, in_place):
    count, past_most, new_most, columns, free_blocks, rows = EXTENDS[case]
    past, more, table, stack = make_requests(case, count, past_most, new_most, columns, free_blocks)
    step, t = run_extend(nv, past, more, table, stack, rows, in_place=in_place, stride=columns + case % 3)
    want = step_ref.extend(past, more, table, list(stack), rows)
    check_extend(step, t, want, table)


@pytest.mark.parametrize("rows", [40, 700, 5000, 20000])
def test_extend_with_too_few_rows_or_blocks_or_columns(nv, rows):
    for seed, (columns, free) in enumerate([(40, 1), (40, 17), (5, 400), (40, 400)]):
        past, more, table, stack = make_requests(seed, 90, 200, 150, columns, free)
        more[3], more[4] = -5, -2**31
        past[5] = columns * BLOCK          # a table that is full
        past[6], more[6] = 2**31 - 10, 50  # a length that ends at 2^31 - 1
        past[7], more[7] = -3, 9           # positions before 0
        step, t = run_extend(nv, past, more, table, stack, rows)
        want = step_ref.extend(past, more, table, list(stack), rows)
        check_extend(step, t, want, table)


@pytest.mark.parametrize("rows", [300, 9000])
def test_extend_with_many_requests_without_rows_between(nv, rows):
    """Rows of one wave that are hundreds of requests apart."""
    count = 3000
    more = [0] * count
    for b, n in ((0, 3), (1, 0), (150, 5), (151, 1), (1200, 2), (2999, 60)):
        more[b] = n
    past, table, stack = [10] * count, [[b, -1] for b in range(count)], list(range(count, count + 9))
    step, t = run_extend(nv, past, more, table, stack, rows)
    check_extend(step, t, step_ref.extend(past, more, table, list(stack), rows), table)


def test_extend_with_a_stack_that_makes_no_sense(nv):
    """A count below 0 or past the capacity stays in bounds: none, or all of the stack."""
    for count, usable in ((-4, 0), (100, 6)):
        free, t = i32([5, 6, 7, 8, 9, 10]), i32([[-1, -1], [-1, -1]])
        step = nv.KvStep.empty(2, 100)
        nv.kv_extend(i32([0, 0]), i32([70, 3]), t, free, i32([count]), step)
        table, stack = [[-1, -1], [-1, -1]], [5, 6, 7, 8, 9, 10][:usable]
        check_extend(step, t, step_ref.extend([0, 0], [70, 3], table, stack, 100), table)


@pytest.mark.parametrize("count,columns,most,keep", [(1, 1, 64, 0), (1, 5, 300, 0), (5, 9, 500, 2), (64, 70, 4400, 0),
                                                     (65, 130, 8000, 3), (700, 200, 9000, 1), (4099, 20, 1200, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_is_the_definition(nv, count, columns, most, keep, in_place):
    lens, _, table, stack = make_requests(count, count, most, 1, columns, 11)
    r = random.Random(count)
    done = [int(r.random() < 0.4) * r.choice([1, -1, 7]) for _ in range(count)]
    done[0] = 1
    for b in range(0, count, 3):  # entries that the pool could not give
        for j in range(0, columns, 4):
            table[b][j] = -1
    if count > 4:
        lens[1], lens[2], lens[3] = 2**31 - 1, -5, 0  # past the table, before 0, nothing held
        done[1] = done[2] = done[3] = 1
        table[1] = list(range(10**6, 10**6 + columns))
    held = sum(-(-max(n, 0) // BLOCK) for n in lens if n < 2**31 - 1) + columns
    for capacity in (len(stack) + held, len(stack) + 3):
        free = i32(stack + [-5] * (capacity - len(stack)))
        n, c, t = i32(lens), i32([len(stack)]), i32(table)
        out = nv.kv_release(n, i32(done), t, free, c, keep=keep, **(dict(lens_out=n, free_count_out=c) if in_place else {}))
        now = list(stack)
        want = step_ref.release(lens, done, table, now, keep, capacity)
        assert out[0].tolist() == want and out[1].tolist() == [len(now)]
        assert free.tolist() == now + [-5] * (capacity - len(now))
        assert t.tolist() == table
        if not in_place:
            assert n.tolist() == lens and c.tolist() == [len(stack)]


def test_a_pool_through_many_steps_in_place(nv):
    """Requests come, grow and finish; no block is held twice or lost."""
    r = random.Random(5)
    count, columns, pool = 40, 12, 300
    past, table, stack = [0] * count, [[-1] * columns for _ in range(count)], list(range(pool))
    lens, free, n_free, t = i32(past), i32(stack), i32([pool]), i32(table)
    step = nv.KvStep.empty(count, 900)
    step.lens, step.free_count = lens, n_free
    for turn in range(30):
        done = [int(r.random() < 0.2) for _ in range(count)]
        more = [r.choice([0, 1, 1, 1, 30, 90]) for _ in range(count)]
        more = [min(m, columns * BLOCK - (0 if d else p)) for m, p, d in zip(more, past, done)]
        nv.kv_release(lens, i32(done), t, free, n_free, lens_out=lens, free_count_out=n_free)
        nv.kv_extend(lens, i32(more), t, free, n_free, step)
        past = step_ref.release(past, done, table, stack, 0, pool)
        want = step_ref.extend(past, more, table, stack, 900)
        check_extend(step, t, want, table)
        past = want["lens"]
        held = [p for b in range(count) for p in table[b][:-(-past[b] // BLOCK)] if p >= 0]
        assert sorted(held + stack) == list(range(pool))
