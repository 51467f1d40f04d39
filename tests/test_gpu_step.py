"""The operators around the cache (norms of heads, tables of a step, attention through a window and over a shared
prefix) against plain references (tests/step_ref.py)."""
import random

import numpy as np
import pytest
import torch

from tests import kv_ref, step_ref
from tests.gpu_util import device
from tests.test_gpu_attention import Pool, bits, check, gen, i32, normal, same, starts, strided, tables_for

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


def test_norm_of_rows_further_apart_than_2_gib(nv):
    """Offsets past 32 bits, in elements and in bytes."""
    far = (1 << 31) + 64
    flat = torch.zeros(2 * far + 512, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(flat, (3, 2, 128), (far, 128, 1))
    host = normal(gen(8), 3, 2, 128)
    x.copy_(host)
    out = torch.as_strided(flat, (3, 2, 128), (far, 128, 1), 256)
    tables = tables_for([64], [9])
    positions = torch.tensor([[8], [0], [5]], dtype=torch.int32)
    nv.norm_rope(x, tables=[t.cuda() for t in tables], positions=positions.cuda(), q_out=out)
    check_norm(out, host, None, 1e-6, tables, positions, False)
    assert same(x, host)


@pytest.mark.parametrize("dim,pairs,split", [(128, [16, 24, 24], False), (128, [24], True), (80, [40], True), (96, [], False)])
def test_norms_of_more_than_the_caches_hold(nv, dim, pairs, split):
    """Outputs past 256 MB, which are stored another way: the bytes of calls on a few rows each."""
    rows, heads, kv_heads = 21001, 50, 9
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    x = torch.randn(rows, heads + kv_heads, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    x = torch.cat([x, x.flip(0)])  # 42,002 rows
    rows = len(x)
    assert x.numel() * 2 > 256 << 20
    size = [31 + 3 * a for a in range(len(pairs))]
    tables = [t.cuda() for t in tables_for(pairs, size)]
    positions = torch.stack([torch.randint(0, n, (rows,), generator=g, device="cuda") for n in size], 1).int() if pairs else None
    w = [torch.randn(dim, generator=g, device="cuda").bfloat16() for _ in range(2)]
    call = lambda a, b: nv.norm_rope(x[a:b, :heads], x[a:b, heads:], *w, tables=tables, split=split,  # noqa: E731
                                     positions=None if positions is None else positions[a:b])
    got = call(0, rows)
    for a in range(0, rows, 7000):
        b = min(rows, a + 7000)
        assert all(torch.equal(y[a:b].view(torch.int16), z.view(torch.int16)) for y, z in zip(got, call(a, b)))
    few = [t.cpu() for t in tables]
    check_norm(got[1][-3:], x[-3:, heads:].cpu(), w[1].cpu(), 1e-6, few, None if positions is None else positions[-3:].cpu(), split)


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
    step = nv.KvStep.empty(n, rows, **(dict(lens=p, free_count=count) if in_place else {}))
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
    (3, 0, 100000, 1700, 5000, 300000), (1026, 100, 9, 3, 2000, 4096), (4093, 100, 9, 3, 9000, 20000),
    (4096, 100, 2, 3, 9000, 4096), (4097, 100, 2, 3, 9000, 4000), (9000, 200, 3, 5, 20000, 30000),
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


@pytest.mark.parametrize("rows", [50, 4500])
def test_extend_into_unaligned_outputs(nv, rows):
    """Positions and slots at any multiple of their elements; what lies beside them is left alone."""
    past, more, table, stack = make_requests(rows, 30, 300, rows // 20, 30, 400)
    want = step_ref.extend(past, more, [list(t) for t in table], list(stack), rows)
    for shift in (1, 2, 3):
        positions = torch.full((rows + 4, 1), -8, dtype=torch.int32, device="cuda")
        slots = torch.full((rows + 4,), -8, dtype=torch.int64, device="cuda")
        other = nv.KvStep.empty(30, rows)
        step = nv.KvStep(other.row_start, other.lens, other.free_count, other.missing, positions[shift:shift + rows],
                         slots[shift:shift + rows], other.workspace)
        nv.kv_extend(i32(past), i32(more), i32(table), i32(stack), i32([len(stack)]), step)
        assert positions.flatten().tolist() == [-8] * shift + want["positions"] + [-8] * (4 - shift)
        assert slots.tolist() == [-8] * shift + want["slots"] + [-8] * (4 - shift)


def test_extend_without_positions_or_slots(nv):
    """Either is left out by the C entry point's null pointer."""
    past, more, table, stack = make_requests(3, 20, 300, 40, 8, 90)
    want = step_ref.extend(past, more, [list(t) for t in table], list(stack), 500)
    for which in ((True, False), (False, True), (False, False)):
        t, free, s = i32(table), i32(stack), nv.KvStep.empty(20, 500)
        s.positions.fill_(-8), s.slots.fill_(-8)
        nv.nvfp4_kv_extend(nv.make_kv_tables(t, free), i32(past), i32(more), i32([len(stack)]), 500, s.row_start, s.lens,
                           s.free_count, s.missing, s.positions if which[0] else None, s.slots if which[1] else None,
                           s.workspace, s.workspace.numel())
        assert s.row_start.tolist() == want["row_start"] and s.lens.tolist() == want["lens"]
        assert s.positions.flatten().tolist() == (want["positions"] if which[0] else [-8] * 500)
        assert s.slots.tolist() == (want["slots"] if which[1] else [-8] * 500)


def test_slots_past_32_bits(nv):
    """Slots of blocks up to the largest number, held and taken."""
    table, stack = [[2**31 - 1, -1, -1], [2**30, 2**25, -1]], [3, 2**25 - 1, 2**25, 2**31 - 1]
    past, more = [10, 100], [100, 60]
    step, t = run_extend(nv, past, more, table, stack, 200)
    check_extend(step, t, step_ref.extend(past, more, table, list(stack), 200), table)
    assert int(step.slots.max()) == (2**31 - 1) * BLOCK + 63


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
    step = nv.KvStep.empty(count, 900, lens=lens, free_count=n_free)
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


# ---------------------------------------------------------------------------
# attention through a window
# ---------------------------------------------------------------------------
# A bound on the lengths decides between 32-row and 128-row tiles and how far the keys are cut; the results have to be
# right with all of them.
BOUND = pytest.mark.parametrize("bound", [None, 0, 1 << 20], ids=["fits", "one-piece", "pieces"])

WINDOWS = [
    # dim, kv heads, group, causal block, window, sinks, [(past, new)]
    (64, 1, 1, 1, 1, 0, [(0, 1)]),
    (128, 1, 1, 1, 1, 1, [(0, 70)]),
    (128, 2, 4, 1, 100, 4, [(516, 1)]),
    (64, 3, 1, 1, 64, 64, [(63, 1), (64, 1), (65, 1), (0, 1), (300, 1)]),
    (128, 2, 5, 1, 63, 1, [(300, 1), (0, 1), (77, 1), (900, 1)]),
    (64, 2, 8, 1, 5, 3, [(100, 3), (10, 2), (0, 3), (5, 0)]),
    (128, 2, 3, 1, 17, 40, [(0, 65), (17, 100)]),
    (64, 2, 2, 0, 30, 0, [(40, 90), (0, 129)]),
    (128, 1, 4, 16, 20, 7, [(5, 60), (64, 48)]),
    (64, 2, 1, 100, 33, 65, [(0, 250)]),
    (128, 3, 1, 0, 129, 2, [(1, 200)]),
    (64, 1, 40, 1, 40, 0, [(70, 3)]),
    (128, 1, 1, 1, 1000, 200, [(3000, 1)]),
    (128, 2, 4, 1, 128, 0, [(0, 400), (333, 200)]),
    (64, 1, 1, 1, 2, 2, [(600, 300)]),
    (64, 2, 7, 1, 200, 130, [(0, 300), (0, 301)]),
    (128, 8, 1, 1, 90, 5, [(0, 300), (77, 130), (0, 0), (500, 65)]),
    (128, 4, 1, 256, 300, 256, [(100, 700)]),
]


@BOUND
@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_window(nv, case, bound):
    dim, heads, group, c, window, sinks, seqs = WINDOWS[case]
    news = [n for _, n in seqs]
    pool = Pool(nv, 250 + case, heads, dim, [p + n for p, n in seqs])
    q = normal(gen(260 + case), sum(news), heads * group, dim, sigma=1.0 + case % 3)
    rs = starts(news)
    want, tol = step_ref.attention(q.double().numpy(), pool.ref, rs, pool.lens.tolist(), pool.table,
                                   np.float64(np.float32(dim ** -0.5)), c, window, sinks)
    call = lambda x, **kw: nv.kv_attention(x, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c, max_len=bound,  # noqa: E731
                                           window=window, sinks=sinks, **kw)
    for layout in ("plain", "qkv", "heads"):
        got = call(strided(q, layout))
        check(got, want, tol)
    out = strided(torch.zeros_like(q), "heads")
    call(q.cuda(), out=out)
    assert same(out, got)
    inplace = q.cuda()
    call(inplace, out=inplace)
    assert same(inplace, got)


@BOUND
@pytest.mark.parametrize("rows", [1, 60, 300])
def test_a_window_past_everything_is_none(nv, bound, rows):
    """What it is without one, and the same bytes however far past everything it reaches where the keys are cut alike,
    which the smaller of the two bounds on what a row sees decides."""
    lens = [900 + rows, 70]
    pool = Pool(nv, 281, 2, 128, lens)
    q = normal(gen(282), rows + 3, 8, 128)
    args = (q.cuda(), pool.gpu, i32([0, rows, rows + 3]), pool.lens, pool.tab)
    exact, tol = step_ref.attention(q.double().numpy(), pool.ref, [0, rows, rows + 3], lens, pool.table,
                                    np.float64(np.float32(128 ** -0.5)), 1)
    check(nv.kv_attention(*args, causal_block=1, max_len=bound), exact, tol)
    first, most = None, pool.tab.shape[1] * BLOCK if bound is None else bound
    for window, sinks in ((2000, 0), (2000, 2000), (1 << 20, 0), (2**31 - 1, 2**31 - 1)):
        got = nv.kv_attention(*args, causal_block=1, max_len=bound, window=window, sinks=sinks)
        check(got, exact, tol)
        if window >= most:
            first = got if first is None else first
            assert same(got, first)


@BOUND
@pytest.mark.parametrize("dim,group,rows,past,window,sinks", [
    (64, 1, 1, 300, 70, 3), (128, 2, 40, 200, 20, 5), (128, 1, 150, 100, 64, 0), (64, 4, 200, 70, 30, 100),
    (128, 2, 3, 2500, 700, 65), (64, 1, 150, 2500, 300, 1), (128, 1, 129, 500, 1, 1)])
def test_what_a_window_hides_has_no_effect(nv, bound, dim, group, rows, past, window, sinks):
    """NaN codes in places that no row sees, and blocks that none sees missing from the table: the outputs' bytes do not
    change.  A NaN that some rows see reaches those rows, and no other."""
    length = past + rows
    pool = Pool(nv, 284, 2, dim, [length])
    q = normal(gen(285), rows, 2 * group, dim)
    call = lambda: nv.kv_attention(q.cuda(), pool.gpu, i32([0, rows]), pool.lens, pool.tab, causal_block=1,  # noqa: E731
                                   max_len=bound, window=window, sinks=sinks)
    clean = call()
    seen = np.stack([step_ref.visible(past + i, length, 1, window, sinks) for i in range(rows)])
    ever = np.concatenate([seen.any(0), np.zeros(-length % BLOCK, bool)])
    for kind in range(2):
        for at in range(len(ever) // BLOCK):
            hidden = ~ever[at * BLOCK:(at + 1) * BLOCK]
            pool.ref.codes[kind][pool.table[0, at]][:, pool.ref.off[kind][hidden]] = 0x7F
    pool.push()
    for at in range(len(ever) // BLOCK):
        if not ever[at * BLOCK:(at + 1) * BLOCK].any():
            pool.tab[0, at] = -3 if at % 2 else 2**31 - 1
    assert same(call(), clean)
    r = random.Random(past)
    for at in {past, length - 1, max(0, past - window), past + rows // 2, max(0, past + 1 - window + rows // 2), 0,
               max(0, sinks - 1), sinks, r.randrange(length)}:
        for kind in range(2):
            if not seen[:, at].any():
                continue
            place = pool.table[0, at // BLOCK], 1, pool.ref.off[kind][at % BLOCK, 3]
            was = pool.ref.codes[kind][place]
            pool.ref.codes[kind][place] = 0xFF
            pool.push()
            got, nan = call().cpu(), torch.zeros(q.shape, dtype=torch.bool)
            i = torch.from_numpy(seen[:, at].nonzero()[0])
            if kind == 0:
                nan[i, group:] = True
            else:
                nan[i, group:, 3] = True
            assert torch.equal(got.isnan(), nan), (at, kind)
            assert np.array_equal(bits(got)[~nan.numpy()], bits(clean)[~nan.numpy()])
            pool.ref.codes[kind][place] = was
    pool.push()
    # a block that some rows see is missing: those rows are NaN, the others as they were
    at = min(length - 1, past + rows // 2) // BLOCK
    pool.tab[0, at] = -1
    nan = torch.from_numpy(seen[:, at * BLOCK:(at + 1) * BLOCK].any(1))
    got = call().cpu()
    assert torch.equal(got.isnan(), nan[:, None, None].expand_as(got))
    assert same(got[~nan], clean.cpu()[~nan])


@BOUND
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_window_rows_that_see_nothing(nv, bound, rows):
    """Sequences of no positions, rows before position 0, a length that the table cannot hold, rows of no sequence."""
    pool = Pool(nv, 286, 1, 64, [0, 5, 70, 64])
    rs = [2, 2 + rows, 2 + 2 * rows, 2 + 3 * rows, 2 + 4 * rows]
    lens = [0, 5, 70, 10**6]
    q = normal(gen(287), rs[-1] + 3, 2, 64)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    nv.kv_attention(q.cuda(), pool.gpu, i32(rs), i32(lens), pool.tab, causal_block=1, out=out, window=20, sinks=3, max_len=bound)
    want, tol = step_ref.attention(q.double().numpy(), pool.ref, rs, lens, pool.table, np.float64(np.float32(0.125)), 1, 20, 3)
    inside = slice(rs[0], rs[-1])
    check(out[inside], want[inside], tol[inside])
    assert bool((out[:rs[0]] == 5).all()) and bool((out[rs[-1]:] == 5).all())
    assert bool((out[rs[0]:rs[1]] == 0).all()) and bool(out[rs[3]:rs[4]].isnan().all())


# ---------------------------------------------------------------------------
# attention over a shared prefix
# ---------------------------------------------------------------------------
SHARED = [
    # dim, kv heads, group, causal block, prefix blocks, [(past behind the prefix, new)]
    (64, 1, 1, 1, 1, [(0, 1)]),
    (128, 1, 1, 1, 1, [(63, 1), (64, 1)]),
    (128, 2, 4, 1, 3, [(16, 1), (0, 1), (100, 1), (5, 1)]),
    (64, 3, 1, 1, 7, [(0, 1), (64, 1), (0, 0), (65, 3), (200, 1)]),
    (64, 2, 8, 1, 2, [(100, 3), (10, 2), (0, 3), (5, 0), (0, 9)]),
    (128, 2, 3, 1, 5, [(0, 65), (17, 100)]),
    (64, 2, 2, 0, 4, [(40, 90), (0, 29)]),
    (128, 1, 4, 16, 2, [(5, 60), (64, 48)]),
    (64, 1, 40, 1, 3, [(70, 3)]),
    (128, 1, 1, 1, 50, [(300, 1), (0, 1)]),
    (128, 8, 1, 1, 3, [(0, 30), (77, 30), (0, 0), (50, 65)]),
    (64, 2, 2, 1, 40, [(i % 9, 1 + i % 2) for i in range(70)]),
]


def shared_pool(nv, seed, heads, dim, blocks, seqs):
    """A pool whose sequences begin with the first one's blocks; the other tables name none there."""
    pool = Pool(nv, seed, heads, dim, [blocks * BLOCK + p + n for p, n in seqs])
    common = pool.table[0, :blocks].copy()
    pool.table[:, :blocks] = -9
    pool.tab = i32(pool.table.tolist())
    return pool, common


@BOUND
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_prefix(nv, case, bound):
    dim, heads, group, c, blocks, seqs = SHARED[case]
    news = [n for _, n in seqs]
    pool, common = shared_pool(nv, 300 + case, heads, dim, blocks, seqs)
    q = normal(gen(310 + case), sum(news) + 5, heads * group, dim, sigma=1.0 + case % 3)
    rs = [3 + r for r in starts(news)]
    want, tol = step_ref.attention(q.double().numpy(), pool.ref, rs, pool.lens.tolist(), pool.table,
                                   np.float64(np.float32(dim ** -0.5)), c, shared=common)
    inside = slice(rs[0], rs[-1])
    call = lambda x, **kw: nv.kv_attention(x, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c, max_len=bound,  # noqa: E731
                                           shared=i32(common.tolist()), **kw)
    for layout in ("plain", "qkv", "heads"):
        got = call(strided(q, layout), out=torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda"))
        check(got[inside], want[inside], tol[inside])
        assert bool((got[:rs[0]] == 5).all()) and bool((got[rs[-1]:] == 5).all())
    out = strided(torch.zeros_like(q), "heads")
    call(q.cuda(), out=out)
    assert same(out[inside], got[inside])
    inplace = q.cuda()
    call(inplace, out=inplace)
    assert same(inplace[inside], got[inside]) and same(inplace[:3], q[:3]) and same(inplace[-2:], q[-2:])


@BOUND
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("blocks,rows,count", [(100, 1, 9), (33, 3, 40), (300, 1, 1), (130, 40, 5)])
def test_a_longer_shared_prefix(nv, bound, dim, blocks, rows, count):
    """Against the sequences' own tables that name the same blocks: one softmax, whatever the pieces."""
    seqs = [(7 * i % 150, rows) for i in range(count)]
    pool, common = shared_pool(nv, 330, 2, dim, blocks, seqs)
    q = normal(gen(331), rows * count, 8, dim).cuda()
    rs = i32(starts([rows] * count))
    got = nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab, causal_block=1, max_len=bound, shared=i32(common.tolist()))
    pool.tab[:, :blocks] = i32(common.tolist())
    want = nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab, causal_block=1).double()
    # each is one rounding of bf16 probabilities (2^-8 of the sums of p |v|, values of order 1) and one of the output
    assert float((got.double() - want).abs().max()) <= 2 * (2.0 ** -8 + 2.0 ** -8) * float(want.abs().max().clamp(min=1))


@BOUND
def test_shared_prefix_errors_of_single_sequences(nv, bound):
    """A sequence whose rows begin inside the prefix, whose length the table cannot hold, or one of whose own blocks is
    missing is NaN, the others as they were; a missing or NaN block of the prefix reaches every row that there is."""
    seqs = [(10, 2), (70, 3), (0, 1), (30, 40)]
    pool, common = shared_pool(nv, 340, 2, 128, 4, seqs)
    q = normal(gen(341), 46, 4, 128).cuda()
    rs, shared = i32([0, 2, 5, 6, 46]), i32(common.tolist())
    call = lambda lens, tab, sh: nv.kv_attention(q, pool.gpu, rs, lens, tab, causal_block=1, max_len=bound, shared=sh).cpu()  # noqa: E731
    clean = call(pool.lens, pool.tab, shared)
    assert bool(clean.isfinite().all())
    for b, length in ((0, 257), (1, 10**6), (2, 0), (1, 258), (3, 255), (3, -1)):
        lens = pool.lens.clone()
        lens[b] = length
        got = call(lens, pool.tab, shared)
        rows = torch.zeros(46, dtype=torch.bool)
        rows[int(rs[b]):int(rs[b + 1])] = True
        assert bool(got[rows].isnan().all()) and same(got[~rows], clean[~rows])
    tab = pool.tab.clone()
    tab[1, 5] = -1
    got = call(pool.lens, tab, shared)
    assert bool(got[2:5].isnan().all())  # position 70 and on: the block of positions 64 .. 127 behind the prefix
    assert same(got[:2], clean[:2]) and same(got[5:], clean[5:])
    for bad in (-1, 10**6):
        assert bool(call(pool.lens, pool.tab, i32([common[0], bad, common[2], common[3]])).isnan().all())
    pool.ref.codes[1][common[2], 1, pool.ref.off[1][5, 9]] = 0x7F
    pool.push()
    got = call(pool.lens, pool.tab, shared)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[:, 2:, 9] = True
    assert torch.equal(got.isnan(), nan) and same(got[~nan], clean[~nan])


def test_a_shared_prefix_of_as_many_rows_as_there_may_be(nv):
    """2^20 sequences of a token and 64 heads, whose joins pass 2^32 threads: 65 keys each, checked where it samples."""
    count, heads, dim = 1 << 20, 64, 64
    pool = Pool(nv, 345, 1, dim, [128])
    g = torch.Generator(device="cuda")
    g.manual_seed(346)
    q = torch.randn(count, heads, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    rs = torch.arange(count + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((count,), BLOCK + 1, dtype=torch.int32, device="cuda")
    table = pool.tab[0, :2].expand(count, 2).contiguous()
    out = nv.kv_attention(q, pool.gpu, rs, lens, table, causal_block=1, shared=pool.tab[0, :1].contiguous())
    sample = torch.tensor([0, 1, 2, 65535, 65536, 262143, 262144, 524288, 999999, count - 2, count - 1], device="cuda")
    n = len(sample)
    want, tol = step_ref.attention(q[sample].cpu().double().numpy(), pool.ref, list(range(n + 1)), [BLOCK + 1] * n,
                                   np.repeat(pool.table, n, 0), np.float64(np.float32(dim ** -0.5)), 1, shared=pool.table[0, :1])
    check(out[sample], want, tol)
    # every row against the same keys in binary32: off by no more than the roundings to bf16 of p, of the sum's p and of o
    k, v = (torch.from_numpy(pool.ref.sequence(kind, 0, pool.table[0], BLOCK + 1)).float().cuda() for kind in range(2))
    most = 0.0
    for i in range(0, count, 1 << 16):
        x = q[i:i + (1 << 16)].reshape(-1, dim).float()
        p = torch.softmax(x @ k.t().contiguous() * dim ** -0.5, 1)
        far = (out[i:i + (1 << 16)].reshape(-1, dim).float() - p @ v).abs() - 3.1 * 2.0 ** -8 * (p @ v.abs())
        most = max(most, float(far.max()))
    assert most <= 0, most


def test_shared_prefix_with_rows_that_make_no_sense_stays_in_bounds(nv):
    pool, common = shared_pool(nv, 342, 1, 64, 2, [(10, 2), (70, 3)])
    q = normal(gen(343), 60, 2, 64).cuda()
    for rs in ([5, 2, 9], [-3, 40, 2000], [0, 0, 0], [60, 60, 60], [2**31 - 1, -2**31, 7], [40, 50, 45]):
        for bound in (None, 0, 1 << 20):
            nv.kv_attention(q, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1, max_len=bound, shared=i32(common.tolist()))
            nv.kv_attention(q, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1, max_len=bound, window=9, sinks=2)
    torch.cuda.synchronize()


def test_a_pool_past_4_gib_through_windows_and_behind_prefixes(nv):
    """Blocks whose offsets pass 32 bits: the same rows through the pool's first and last blocks."""
    heads, dim, n = 8, 128, 200
    blocks = 2**32 // (heads * 64 * dim) + 100  # 4 GiB of keys and as much of values
    pool = nv.KvCache.empty(blocks, heads, dim)
    g = gen(7)
    k, v, q = (normal(g, n, h, dim).cuda() for h in (heads, heads, 2 * heads))
    rs, lens = i32([0, n]), i32([n])
    got = []
    for table in ([0, 1, 2, 3], [blocks - 1, blocks - 90, blocks - 2, blocks - 50]):
        tab, few = i32([table]), i32([0, 5])
        nv.kv_write(pool, k, v, rs, lens, tab)
        got.append([nv.kv_attention(x, pool, r, lens, tab, causal_block=1, **kw) for x, r in ((q, rs), (q[-5:], few))
                    for kw in (dict(window=70, sinks=3), dict(shared=tab[0, :1].contiguous()), dict(shared=tab[0, :3].contiguous()))
                    if not (r is rs and "shared" in kw)])
    for a, b in zip(*got):
        assert same(a, b) and bool(a.isfinite().all())


@pytest.mark.parametrize("rows", [1, 40, 130])
def test_a_window_at_the_end_of_the_longest_sequence(nv, rows):
    """Positions up to 2^31 - 65 in a table that names one block throughout: the bytes of a short sequence of it."""
    pool = Pool(nv, 290, 2, 64, [BLOCK])
    q = normal(gen(291), rows, 4, 64).cuda()
    got = []
    for blocks in ((1 << 25) - 1, 101):
        table = torch.full((1, blocks), int(pool.table[0, 0]), dtype=torch.int32, device="cuda")
        for window, sinks, c in ((1000, 5, 1), (1, 0, 1), (500, 100, 64), (77, 0, 0)):
            got.append(nv.kv_attention(q, pool.gpu, i32([0, rows]), i32([blocks * BLOCK]), table, causal_block=c, window=window,
                                       sinks=sinks, max_len=6464))
    for a, b in zip(got[:4], got[4:]):
        assert same(a, b) and bool(a.isfinite().all())


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Serving:
    """A few requests over one pool: what a program keeps from step to step, and one step of it."""

    def __init__(self, nv, shared_blocks=0):
        self.nv, self.count, self.heads, self.dim, self.rows, self.pool = nv, 5, 2, 128, 130, 64
        self.cache = nv.KvCache.empty(self.pool, self.heads, self.dim)
        self.table = torch.full((self.count, 12), -1, dtype=torch.int32, device="cuda")
        self.shared = i32(list(range(shared_blocks))) if shared_blocks else None
        self.keep = shared_blocks
        if shared_blocks:
            g = gen(77)
            n = shared_blocks * BLOCK
            k, v = normal(g, n, self.heads, self.dim).cuda(), normal(g, n, self.heads, self.dim).cuda()
            nv.kv_write(self.cache, k, v, i32([0, n]), i32([n]), self.shared[None])
            self.table[:, :shared_blocks] = self.shared
        self.lens = i32([shared_blocks * BLOCK] * self.count)
        self.free = i32(list(range(shared_blocks, self.pool)))
        self.n_free = i32([self.pool - shared_blocks])
        self.step_arrays = nv.KvStep.empty(self.count, self.rows, lens=self.lens, free_count=self.n_free)
        self.tables = [nv.rope_table(2048, 64)]
        g = gen(78)
        self.weights = [(1 + normal(g, self.dim, sigma=0.1).float()).bfloat16().cuda() for _ in range(2)]
        self.more, self.done = i32([0] * self.count), i32([0] * self.count)
        self.base = i32([shared_blocks * BLOCK] * self.count)
        self.x = torch.zeros(self.rows, 12, self.dim, dtype=torch.bfloat16, device="cuda")
        # rows of no request are not written by the attention, and the quantizer's one scale is that of all rows
        self.o = torch.zeros(self.rows, 4 * self.heads, self.dim, dtype=torch.bfloat16, device="cuda")

    def step(self):
        nv, h = self.nv, self.heads
        nv.kv_release(self.lens, self.done, self.table, self.free, self.n_free, keep=self.keep, lens_out=self.lens,
                      free_count_out=self.n_free)
        torch.maximum(self.lens, self.base, out=self.lens)  # a new request begins behind the prefix
        s = nv.kv_extend(self.lens, self.more, self.table, self.free, self.n_free, self.step_arrays)
        q, k = nv.norm_rope(self.x[:, :4 * h], self.x[:, 4 * h:5 * h], *self.weights, tables=self.tables, positions=s.positions,
                            split=True)
        nv.kv_write(self.cache, k, self.x[:, 5 * h:], s.row_start, s.lens, self.table)
        if self.shared is not None:
            nv.kv_attention(q, self.cache, s.row_start, s.lens, self.table, causal_block=1, shared=self.shared, out=self.o)
        else:
            nv.kv_attention(q, self.cache, s.row_start, s.lens, self.table, causal_block=1, window=100, sinks=4, out=self.o)
        return nv.quantize(self.o.reshape(self.rows, -1))


@pytest.mark.parametrize("shared", [0, 3])
def test_a_serving_step_eager_and_captured(nv, shared):
    """Release, extend, norms and rotation, cache, attention, quantizer: eager steps against the references, and the same
    step captured once and replayed with new inputs, eager work between: every replay equals the eager step."""
    eager, captured = Serving(nv, shared), Serving(nv, shared)
    side = torch.cuda.Stream()
    Serving(nv, shared).step()  # what a first call sets up stays out of the capture
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        graph_out = captured.step()
    r, g = random.Random(shared), gen(79)
    ref = kv_ref.Cache(eager.pool, eager.heads, eager.dim)
    for c, t in zip(ref.codes + ref.powers, (eager.cache.k, eager.cache.v, eager.cache.k_power, eager.cache.v_power)):
        c[:] = t.cpu().numpy().reshape(c.shape)
    lens = [shared * BLOCK] * 5
    table, stack = eager.table.tolist(), eager.free.tolist()
    tables = [t.cpu() for t in eager.tables]
    weights = [w.cpu() for w in eager.weights]
    for turn in range(6):
        x = normal(g, eager.rows, 12, eager.dim)
        done = [int(turn > 1 and r.random() < 0.3) for _ in range(5)]
        more = [r.choice([1, 1, 20, 40, 0]) for _ in range(5)]
        for s in (eager, captured):
            s.x.copy_(x), s.done.copy_(i32(done)), s.more.copy_(i32(more))
        out = [t.clone() for t in eager.step()]
        graph.replay()
        torch.cuda.synchronize()
        now = step_ref.release(lens, done, table, stack, shared, eager.pool - shared)
        now = [max(n, shared * BLOCK) for n in now]
        want = step_ref.extend(now, more, table, stack, eager.rows)
        lens, rs = want["lens"], want["row_start"]
        assert eager.lens.tolist() == lens and eager.table.tolist() == table and eager.n_free.tolist() == [len(stack)]
        used = rs[-1]
        positions = torch.tensor(want["positions"], dtype=torch.int32)[:, None]
        q, k = (step_ref.norm_rope(x[:used, a:b], w, 1e-6, tables, positions[:used], True)[0]
                for a, b, w in ((0, 8, weights[0]), (8, 10, weights[1])))
        # what the kernels themselves made of the rows goes on: the cache as it stands, the queries as they were rounded
        for c, t in zip(ref.codes + ref.powers, (eager.cache.k, eager.cache.v, eager.cache.k_power, eager.cache.v_power)):
            c[:] = t.cpu().numpy().reshape(c.shape)
        made = nv.norm_rope(eager.x[:, :8], None, eager.weights[0], tables=eager.tables, positions=eager.step_arrays.positions,
                            split=True).cpu()
        assert float((made[:used].double() - q).abs().max()) <= 2.0 ** -8 * float(q.abs().max()) * 1.01
        for b in range(5):  # keys in the cache: 8-bit codes of the normed ones (2^-4 of the value, 2^-10 of the block's largest)
            for h in range(2):
                held = ref.sequence(0, h, np.array(table[b]), lens[b])[lens[b] - (rs[b + 1] - rs[b]):]
                mine = k[rs[b]:rs[b + 1], h].numpy()
                if len(mine):
                    assert np.all(np.abs(held - mine) <= 2.0 ** -3 * np.abs(mine) + 2.0 ** -8 * float(k.abs().max()))
        o, tol = step_ref.attention(made.double().numpy(), ref, rs, lens, np.array(table), np.float64(np.float32(128 ** -0.5)), 1,
                                    *((0, 0) if shared else (100, 4)), shared=np.arange(shared) if shared else None)
        check(eager.o[:used], o[:used], tol[:used])
        assert all(torch.equal(a, b) for a, b in zip(out, graph_out)) and bool(out[2].isfinite().all()), f"replay {turn}"
        assert same(eager.o[:used], captured.o[:used]), f"replay {turn}"
        for name in ("lens", "table", "n_free", "free"):
            assert torch.equal(getattr(eager, name), getattr(captured, name)), name
        for a, b in ((eager.cache.k, captured.cache.k), (eager.cache.v, captured.cache.v)):
            assert torch.equal(a, b)


def test_norms_and_tables_on_other_streams(nv):
    """On a side stream that is given or current, behind work that is still running there: what they give on the main one."""
    x = normal(gen(360), 300, 6, 128).cuda()
    past, more, table, stack = make_requests(361, 30, 300, 40, 9, 90)
    want = step_ref.extend(past, more, [list(t) for t in table], list(stack), 900)
    norm = nv.norm_rope(x)
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for given in (True, False):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(20):
                y = big @ big
            late = x + 0 * y[:300, :1, None].bfloat16().nan_to_num(0)
            p, t, free, n = i32(past), i32(table), i32(stack), i32([len(stack)])
        kw = dict(stream=side) if given else {}
        with torch.cuda.stream(torch.cuda.current_stream() if given else side):
            got = nv.norm_rope(late, **kw)
            step = nv.kv_extend(p, i32(more) if not given else more_on(side, more), t, free, n, nv.KvStep.empty(30, 900, **kw), **kw)
        side.synchronize()
        assert same(got, norm)
        assert step.slots.tolist() == want["slots"] and step.lens.tolist() == want["lens"]


def more_on(side, more):
    with torch.cuda.stream(side):
        return i32(more)


@pytest.mark.parametrize("kw", [dict(window=200, sinks=5), "shared"])
def test_other_streams_and_the_same_bytes(nv, kw):
    """Calls on side streams, two at once with workspaces of their own, equal the calls on the main one."""
    pool, common = shared_pool(nv, 350, 2, 128, 20, [(700, 1), (50, 1)])
    if kw == "shared":
        kw = dict(shared=i32(common.tolist()))
    else:
        pool.tab[:, :20] = i32(common.tolist())
    q = normal(gen(351), 2, 8, 128).cuda()
    rs = i32([0, 1, 2])
    want = nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab, causal_block=1, **kw)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in side:
            got.append(nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab, causal_block=1, stream=s, **kw))
    for s in side:
        s.synchronize()
    for o in got:
        assert same(o, want)


# ---------------------------------------------------------------------------
# no rows, no requests
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("requests,rows", [(3, 0), (0, 5), (0, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_of_no_rows_or_no_requests(nv, requests, rows, in_place):
    """What the definition gives: nothing.  Also captured, and on a stream that is given."""
    past, more, stack = [7, 64, -3][:requests], [4, 90, 0][:requests], [4, 5, 6]
    table = torch.full((requests, 4), -1, dtype=torch.int32, device="cuda")
    for count, free_after in ((3, 3), (-2, 0), (9, 5)):
        n, c, free = i32(past), i32([count]), i32(stack + [-5, -5])
        step = nv.KvStep.empty(requests, rows, **(dict(lens=n, free_count=c) if in_place else {}))
        asked, side = i32(more), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv.kv_extend(n, asked, table, free, c, step)
        for how in range(3):
            step.row_start.fill_(9), step.missing.fill_(9), step.positions.fill_(9), step.slots.fill_(9)
            if how == 0:
                assert nv.kv_extend(n, asked, table, free, c, step) is step
            elif how == 1:
                side.wait_stream(torch.cuda.current_stream())
                nv.kv_extend(n, asked, table, free, c, step, stream=side)
                side.synchronize()
            else:
                graph.replay()
                torch.cuda.synchronize()
            want = step_ref.extend(past, more, table.tolist() or [[]], list(range(free_after)), rows)
            check_extend(step, table, want, table.tolist())
            assert n.tolist() == past and free.tolist() == stack + [-5, -5] and int(table.max()) == -1 if requests else True


def test_release_of_no_requests(nv):
    none, table = i32([]), torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    for count, after in ((2, 2), (-4, 0), (8, 3)):
        free = i32([1, 2, -5])
        lens, left = nv.kv_release(none, none, table, free, i32([count]))
        assert lens.shape == (0,) and left.tolist() == [after] and free.tolist() == [1, 2, -5]
        c = i32([count])
        assert nv.kv_release(none, none, table, free, c, free_count_out=c, to_prefix=True)[1] is c and c.tolist() == [after]
    with pytest.raises(TypeError, match="done: expected int32"):
        nv.kv_release(none, none.long(), table, i32([1]), i32([1]))
    with pytest.raises(ValueError, match="a table of 0 requests, a step of 2"):
        nv.kv_extend(none, none, table, i32([1]), i32([1]), nv.KvStep.empty(2, 3))


# ---------------------------------------------------------------------------
# requests behind a prefix that stays
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("count,keep", [(1, 1), (5, 3), (40, 2), (700, 1)])
def test_a_pool_behind_a_prefix_through_many_steps_in_place(nv, count, keep):
    """Requests come, grow and finish behind kept blocks: no block is held twice or lost, the tables go on naming the
    prefix, and new rows begin behind it."""
    r = random.Random(count)
    columns, own = keep + 6, 4 * count
    prefix, stack = list(range(keep)), list(range(keep, keep + own))
    table = [prefix + [-1] * 6 for _ in range(count)]
    past = [keep * BLOCK] * count
    lens, free, n_free, t = i32(past), i32(stack), i32([own]), i32(table)
    rows = 130 * count
    step = nv.KvStep.empty(count, rows, lens=lens, free_count=n_free)
    for turn in range(12):
        done = [int(r.random() < 0.4) for _ in range(count)]
        now = [keep * BLOCK if d else p for d, p in zip(done, past)]
        more = [min(r.choice([0, 1, 1, 30, 130]), columns * BLOCK - p) for p in now]
        nv.kv_release(lens, i32(done), t, free, n_free, keep=keep, lens_out=lens, free_count_out=n_free, to_prefix=True)
        step_ref.release(past, done, table, stack, keep, own)
        assert lens.tolist() == now and n_free.tolist() == [len(stack)]
        nv.kv_extend(lens, i32(more), t, free, n_free, step)
        want = step_ref.extend(now, more, table, stack, rows)
        check_extend(step, t, want, table)
        past = want["lens"]
        held = [p for b in range(count) for p in table[b][keep:-(-past[b] // BLOCK)] if p >= 0]
        assert sorted(held + stack) == list(range(keep, keep + own))
        assert all(row[:keep] == prefix for row in table)


@pytest.mark.parametrize("count,columns", [(3, 4), (99, 7)])
def test_lengths_of_what_is_released_to_a_prefix(nv, count, columns):
    """64 * keep, at most what the table holds; the others' as they were; blocks as without it."""
    lens, _, table, stack = make_requests(count, count, columns * BLOCK, 1, columns, 3)
    done = [b % 3 == 0 for b in range(count)]
    for keep in (0, 1, columns, columns + 1, 2**31 - 1):
        free = [i32(stack + [-5] * (count * columns)) for _ in range(2)]
        out = [nv.kv_release(i32(lens), i32(done), i32(table), f, i32([len(stack)]), keep=keep, to_prefix=to)
               for f, to in zip(free, (False, True))]
        assert torch.equal(*free) and torch.equal(out[0][1], out[1][1])
        assert out[1][0].tolist() == [min(keep, columns) * BLOCK if d else n for d, n in zip(done, lens)]


# ---------------------------------------------------------------------------
# rows of no request
# ---------------------------------------------------------------------------
KINDS = ["plain", "window", "shared"]


def kind_args(kind, common):
    return {"plain": {}, "window": dict(window=50, sinks=3), "shared": dict(shared=common)}[kind]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,heads,group,rows,layout", [(64, 1, 1, 1, "plain"), (128, 2, 4, 67, "qkv"), (64, 3, 5, 300, "heads"),
                                                         (128, 1, 70, 9, "plain")])
def test_rows_of_no_sequence_are_cleared(nv, kind, dim, heads, group, rows, layout):
    """And no others: the sequences' rows have the bytes of a call without it, what lies beside the output is untouched.
    Row starts that make no sense stay in bounds."""
    pool = Pool(nv, 370, heads, dim, [200 + rows, 200 + rows])
    pool.tab[1, 0] = pool.tab[0, 0]
    common = pool.tab[0, :1].contiguous()
    q = normal(gen(371), rows, heads * group, dim).cuda()
    for rs in ([0, 0, 0], [0, rows // 2, rows], [rows // 3, rows // 2, rows - rows // 4], [rows, rows, rows], [0, 0, 1],
               [rows - 1, rows, rows], [-5, 1, rows + 9], [2**31 - 1, 0, -2**31], [5, 2, 1]):
        call = lambda x, **kw: nv.kv_attention(x, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1,  # noqa: E731
                                               **kind_args(kind, common), **kw)
        first = min(max(rs[0], 0), rows)
        last = min(max(rs[2], first), rows)
        made = strided(torch.full_like(q, 5.0), layout)
        call(q, out=made)
        out = strided(torch.full_like(q, float("nan")), layout)
        assert call(q, out=out, clear_rest=True) is out
        rest = torch.ones(rows, dtype=torch.bool, device="cuda")
        rest[first:last] = False
        assert bool((made[rest] == 5).all()) and bool((out.view(torch.int16)[rest] == 0).all())
        if sorted(rs) == rs:
            assert same(out[~rest], made[~rest])
        if layout == "qkv":
            wide = torch.as_strided(out, (rows, 3 * heads * group, dim), (3 * heads * group * dim, dim, 1), 0)
            assert bool((wide[:, :heads * group] == 7).all()) and bool((wide[:, 2 * heads * group:] == 7).all())


def test_clearing_rows_further_apart_than_2_gib(nv):
    """Offsets past 32 bits, and more rows than workgroups."""
    far = (1 << 31) + 64
    flat = torch.ones(2 * far + 512, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(flat, (3, 2, 128), (far, 128, 1))
    nv.nvfp4_kv_clear_rest(nv.make_heads("out", out), 3, 2, 128, i32([1, 2]), 1)
    assert bool((out[[0, 2]] == 0).all()) and bool((out[1] == 1).all())
    assert int((flat == 0).sum()) == 2 * 2 * 128
    many = torch.ones(5000, 1, 16, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_kv_clear_rest(nv.make_heads("out", many), 5000, 1, 16, i32([2001, 2001, 2004]), 2)
    assert (many[:, 0, :] == 1).all(1).nonzero().flatten().tolist() == [2001, 2002, 2003] and int((many == 0).sum()) == 4997 * 16


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["kept", "new", "queries"])
def test_rows_of_no_request_do_not_reach_the_quantizer(nv, kind, where):
    """Steps of few rows after one of many and large ones, eager and replayed: the quantizer's scale and codes are those of
    the rows in use, whichever output the attention writes."""
    rows, heads, dim = 130, 2, 128
    cache, common = nv.KvCache.empty(30, heads, dim), i32([0])
    table = i32([[0] + list(range(1, 8)), [0] + list(range(8, 15))])
    prefix = normal(gen(380), BLOCK, heads, dim, sigma=0.1).cuda()
    nv.kv_write(cache, prefix, prefix, i32([0, BLOCK]), i32([BLOCK]), common[None])
    x = torch.zeros(rows, 12, dim, dtype=torch.bfloat16, device="cuda")
    base, more, free, n_free = i32([BLOCK, BLOCK]), i32([0, 0]), i32(list(range(15, 30))), i32([15])
    step = nv.KvStep.empty(2, rows)
    o, tables = torch.zeros(rows, 8, dim, dtype=torch.bfloat16, device="cuda"), [nv.rope_table(1024, 64)]

    def run():
        s = nv.kv_extend(base, more, table, free, n_free, step)
        q, k = nv.norm_rope(x[:, :8], x[:, 8:10], tables=tables, positions=s.positions, split=True)
        nv.kv_write(cache, k, x[:, 10:], s.row_start, s.lens, table)
        out = nv.kv_attention(q, cache, s.row_start, s.lens, table, causal_block=1, clear_rest=True, **kind_args(kind, common),
                              **{"kept": dict(out=o), "new": {}, "queries": dict(out=q)}[where])
        return (out, *nv.quantize(out.reshape(rows, -1)))

    run()  # what a first call sets up stays out of the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = run()
    for turn, (counts, size) in enumerate([((100, 30), 50.0), ((1, 1), 1.0), ((0, 3), 0.5), ((70, 60), 20.0), ((0, 0), 1.0),
                                           ((5, 0), 2.0)]):
        dirt = torch.full((200, 8, dim), float("nan"), dtype=torch.bfloat16, device="cuda")  # what a new output may hold
        del dirt
        x.copy_(normal(gen(381 + turn), rows, 12, dim))
        x[:, 10:] *= size
        more.copy_(i32(list(counts)))
        used = sum(counts)
        for got in (run(), None):
            if got is None:
                graph.replay()
                torch.cuda.synchronize()
                got = replayed
            out, codes, scales, tensor_scale, amax = got
            assert bool((out[used:] == 0).all()) and bool(out.isfinite().all())
            assert float(amax) == float(out[:used].abs().max() if used else 0), (turn, used)
            if used:
                alone = nv.quantize(out[:used].reshape(used, -1).contiguous())
                assert torch.equal(alone[0][:used], codes[:used]) and torch.equal(alone[2], tensor_scale)
