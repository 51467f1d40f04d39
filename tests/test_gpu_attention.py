"""Rotary positions, the 8-bit key/value cache and attention over it, against plain references (tests/kv_ref.py)."""
import functools
import types

import numpy as np
import pytest
import torch

from tests import kv_ref
from tests.gpu_util import device

pytestmark = pytest.mark.gpu
BLOCK = 64


@pytest.fixture(scope="module")
def nv(request):
    import nvfp4_activation_quantization_segment_amd as m

    device()
    bound = getattr(request, "param", None)
    if bound is None:
        return m
    return types.SimpleNamespace(**dict(vars(m), kv_attention=functools.partial(m.kv_attention, max_len=bound)))


# The bound on the lengths decides between 32-row and 128-row tiles and how far the keys are cut: what the table
# holds mostly gives 32 rows at these sizes, 0 gives 128 rows in one piece (from 64 rows a sequence on), a large
# one 128 rows in many pieces.  The results have to be right with all of them.
BOUNDS = pytest.mark.parametrize("nv", [None, 0, 1 << 20], indirect=True, ids=["fits", "one-piece", "pieces"])


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g) * sigma).to(torch.bfloat16)


def bits(t):
    return t.contiguous().cpu().view(torch.int16).numpy()


def same(a, b):
    """Whether two bf16 tensors hold the same bits."""
    return bool((bits(a) == bits(b)).all())


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def strided(x, layout):
    """x [rows, heads, dim] on the GPU in another layout, same values."""
    rows, heads, dim = x.shape
    if layout == "qkv":  # the middle of a wider product
        wide = torch.full((rows, 3 * heads, dim), 7.0, dtype=x.dtype, device="cuda")
        wide[:, heads:2 * heads] = x.cuda()
        return wide[:, heads:2 * heads]
    if layout == "heads":  # [heads, rows, dim]
        return x.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    return x.cuda()


def tables_for(pairs, size, theta=100.0):
    got = []
    for n, p in zip(size, pairs):
        angle = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-torch.arange(p, dtype=torch.float64) / p)
        got.append(torch.stack([angle.cos(), angle.sin()], -1).float())
    return got


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,heads,dim,pairs,split,layout", [
    (1, 1, 64, [32], False, "plain"),
    (1, 1, 16, [8], True, "plain"),
    (5, 3, 64, [8, 8, 16], False, "qkv"),
    (5, 3, 64, [22, 5, 5], True, "heads"),
    (129, 56, 128, [16, 24, 24], False, "qkv"),
    (67, 56, 128, [22, 21, 21], True, "qkv"),
    (33, 7, 128, [32], True, "plain"),
    (33, 33, 128, [1, 1, 1, 13], False, "heads"),
    (19, 5, 80, [40], False, "plain"),
    (3, 300, 64, [16], True, "plain"),
    (2, 2, 512, [100, 100], False, "plain"),
    (300, 1, 96, [24, 16], True, "qkv"),
    (8195, 40, 64, [8, 12, 12], False, "plain"),  # several rows to a workgroup although one fills it
    (8192, 20, 64, [24], True, "qkv"),
])
def test_rope_is_the_formula_bit_for_bit(nv, rows, heads, dim, pairs, split, layout):
    g = gen(rows * dim + heads)
    x = normal(g, rows, heads, dim)
    size = [11 + 3 * a for a in range(len(pairs))]
    tables = tables_for(pairs, size)
    positions = torch.stack([torch.randint(0, n, (rows,), generator=g) for n in size], 1).int()
    want = kv_ref.rotate(x, tables, positions, split)
    xs = strided(x, layout)
    got = nv.rope(xs, [t.cuda() for t in tables], positions.cuda(), split=split)
    assert same(got, want.to(torch.bfloat16))
    # against the formula in 64 bits: two products and a sum in binary32, then bf16
    exact = kv_ref.rotate(x, tables, positions, split, torch.float64)
    # each output is a sum of two products of an element and a cosine or sine, so at most 2 amax
    amax = float(x.abs().max())
    assert float((got.cpu().double() - exact).abs().max()) <= 2 * amax * (2.0 ** -8 + 4 * 2.0 ** -24)
    out = strided(torch.zeros_like(x), layout)
    assert nv.rope(xs, [t.cuda() for t in tables], positions.cuda(), split=split, out=out) is out
    assert same(out, got)
    if layout == "qkv":  # what lies beside the heads is untouched, also in place
        nv.rope(xs, [t.cuda() for t in tables], positions.cuda(), split=split, out=xs)
        wide = xs._base if xs._base is not None else xs
        assert same(xs, got)
        wide = torch.as_strided(xs, (rows, 3 * heads, dim), (3 * heads * dim, dim, 1), 0)
        assert bool((wide[:, :heads] == 7).all()) and bool((wide[:, 2 * heads:] == 7).all())


def test_rope_leaves_the_other_dims_and_marks_bad_positions(nv):
    x = normal(gen(1), 6, 2, 128)
    x[..., 64:] = torch.tensor([float("nan"), float("inf"), -0.0, float("-inf")] * 16, dtype=torch.bfloat16)
    tables = [t.cuda() for t in tables_for([16, 16], [5, 7])]
    positions = torch.tensor([[0, 0], [4, 6], [5, 0], [0, 7], [-1, 0], [2**31 - 1, -2**31]], dtype=torch.int32)
    for split in (False, True):
        got = nv.rope(x.cuda(), tables, positions.cuda(), split=split).cpu()
        assert same(got[..., 64:], x[..., 64:])
        good = kv_ref.rotate(x[:2], [t.cpu() for t in tables], positions[:2], split).to(torch.bfloat16)
        assert same(got[:2, :, :64], good[..., :64])
        nan = got[..., :64].isnan()
        by_axis = torch.zeros(64, dtype=torch.int64)
        for i in range(32):
            p, q = (i, i + 32) if split else (2 * i, 2 * i + 1)
            by_axis[p] = by_axis[q] = i // 16
        bad = torch.tensor([[False, False], [False, False], [True, False], [False, True], [True, False], [True, True]])
        assert torch.equal(nan, bad[:, by_axis][:, None, :].expand(-1, 2, -1))


def test_rope_table(nv):
    t = nv.rope_table(5000, 21, theta=10000.0).cpu().double()
    angle = torch.arange(5000, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(21, dtype=torch.float64) / 21)
    want = torch.stack([angle.cos(), angle.sin()], -1)
    # binary64 angles (an error of a few 2^-53 of up to 5000) rounded once to binary32, values at most 1
    assert float((t - want).abs().max()) <= 2.0 ** -25 + 5000 * 8 * 2.0 ** -53
    assert tuple(nv.rope_table(1, 1).shape) == (1, 1, 2)


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
class Pool:
    """A GPU cache and the same pool on the host, filled with the same bytes."""

    def __init__(self, nv, seed, heads, dim, lens, spare=2, filled=True):
        g = gen(seed)
        self.heads, self.dim = heads, dim
        need = [max(1, -(-n // BLOCK)) for n in lens]
        blocks = sum(need) + spare
        order = torch.randperm(blocks, generator=g).tolist()
        self.table = np.full((len(lens), max(need)), -7, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.ref = kv_ref.Cache(blocks, heads, dim)
        if filled:
            r = np.random.RandomState(seed)
            for kind in range(2):
                self.ref.codes[kind][:] = r.randint(0, 256, self.ref.codes[kind].shape)
                c = self.ref.codes[kind]
                c[(c & 0x7F) == 0x7F] = 0x30  # no NaN codes
                # codes of |value| up to 448 with powers about 2^-8: values of order 1
                self.ref.powers[kind][:] = 118 + r.randint(0, 4, self.ref.powers[kind].shape)
        self.gpu = nv.KvCache.empty(blocks, heads, dim)
        self.push()
        self.lens = i32(lens)
        self.tab = i32(self.table.tolist())

    def push(self):
        for t, a in ((self.gpu.k, self.ref.codes[0]), (self.gpu.v, self.ref.codes[1]),
                     (self.gpu.k_power, self.ref.powers[0]), (self.gpu.v_power, self.ref.powers[1])):
            t.copy_(torch.from_numpy(a).reshape(t.shape))

    def pulled(self):
        return [t.cpu().numpy().reshape(a.shape) for t, a in
                ((self.gpu.k, self.ref.codes[0]), (self.gpu.v, self.ref.codes[1]),
                 (self.gpu.k_power, self.ref.powers[0]), (self.gpu.v_power, self.ref.powers[1]))]

    def same(self):
        for got, want, name in zip(self.pulled(), self.ref.codes + self.ref.powers, ("k", "v", "k_power", "v_power")):
            if name in "kv":  # the sign of a NaN code is free
                got, want = (np.where((a & 0x7F) == 0x7F, 0x7F, a) for a in (got, want))
            bad = np.argwhere(got != want)
            assert bad.size == 0, f"{name}: {len(bad)} bytes differ, first at {bad[0]}: {got[tuple(bad[0])]} for " \
                                  f"{want[tuple(bad[0])]}"


def starts(news):
    return [0] + np.cumsum(news).tolist()


WRITES = [
    # heads, dim, [(past, new)]
    (1, 64, [(0, 1)]),
    (1, 128, [(0, 64)]),
    (3, 128, [(0, 200)]),
    (2, 64, [(0, 129), (0, 0), (0, 63)]),
    (2, 128, [(63, 1), (64, 1), (65, 1), (0, 1)]),
    (2, 64, [(1, 62), (1, 63), (1, 64), (1, 200)]),
    (9, 64, [(37, 5), (0, 0), (130, 3), (190, 70)]),
    (17, 128, [(77, 301), (5, 3)]),
    # at most one row a sequence on average, and at most four: the short writer
    (5, 128, [(63, 1), (0, 1), (64, 1), (150, 1), (7, 0), (200, 1)]),
    (2, 64, [(100, 150)] + [(i, 0) for i in range(150)]),
    (3, 128, [(30, 100)] + [(i, 1) for i in range(40)]),
    (2, 64, [(60, 9), (126, 3), (0, 2), (5, 1), (64, 4)]),
]


@pytest.mark.parametrize("case", range(len(WRITES)))
@pytest.mark.parametrize("layout", ["plain", "qkv", "heads"])
def test_kv_write_is_the_formula_byte_for_byte(nv, case, layout):
    heads, dim, seqs = WRITES[case]
    news = [n for _, n in seqs]
    pool = Pool(nv, 10 + case, heads, dim, [p + n for p, n in seqs])
    g = gen(100 + case)
    k, v = normal(g, sum(news), heads, dim), normal(g, sum(news), heads, dim, sigma=0.01)
    # heads of very different sizes, so that some blocks' powers grow and others' do not
    k *= torch.exp2(torch.randint(-9, 10, (1, heads, 1), generator=g).float()).to(torch.bfloat16)
    rs = starts(news)
    pool.ref.write((k.double().numpy(), v.double().numpy()), rs, pool.lens.tolist(), pool.table)
    nv.kv_write(pool.gpu, strided(k, layout), strided(v, layout), i32(rs), pool.lens, pool.tab)
    pool.same()
    # written again, the cache holds the same
    nv.kv_write(pool.gpu, strided(k, layout), strided(v, layout), i32(rs), pool.lens, pool.tab)
    pool.same()


def test_kv_write_of_many_heads_and_blocks(nv):
    """More heads than one workgroup takes at once, so that the loop over heads runs (56 heads of 700 positions)."""
    heads, dim, n = 56, 64, 4000
    pool = Pool(nv, 5, heads, dim, [n], filled=False)
    g = gen(6)
    k, v = normal(g, n, heads, dim), normal(g, n, heads, dim)
    nv.kv_write(pool.gpu, k.cuda(), v.cuda(), i32([0, n]), pool.lens, pool.tab)
    pool.ref.write((k.double().numpy(), v.double().numpy()), [0, n], [n], pool.table)
    pool.same()


def test_kv_write_of_special_values(nv):
    """Zeros, the smallest and largest magnitudes, infinities and NaN, in blocks of their own and beside others."""
    dim, heads = 64, 6
    pool = Pool(nv, 3, heads, dim, [130])
    k = normal(gen(4), 130, heads, dim)
    k[:, 0] = 0.0
    k[:, 1] = 2.0 ** -133
    k[5, 1, 3] = -(2.0 ** -130)
    k[:, 2] = torch.finfo(torch.bfloat16).max
    k[3, 3, 5], k[70, 3, 6], k[128, 3, 0] = float("inf"), float("-inf"), float("nan")
    k[:, 4] = float("nan")
    k[:, 5, ::2], k[:, 5, 1::2] = -0.0, 448.0
    v = k.flip(1)
    rows = (k.double().numpy(), v.double().numpy())
    nv.kv_write(pool.gpu, k.cuda(), v.cuda(), i32([0, 130]), pool.lens, pool.tab)
    pool.ref.write(rows, [0, 130], [130], pool.table)
    pool.same()
    # and back: code times power, NaN where the value was not finite
    back = nv.kv_read(pool.gpu, 130, i32([0, 130]), pool.lens, pool.tab)
    for kind in range(2):
        for h in range(heads):
            want = pool.ref.sequence(kind, h, pool.table[0], 130)
            assert np.array_equal(back[kind][:, h].cpu().double().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("rows", [1, 3])
def test_short_write_of_special_values(nv, rows):
    """The special values one or three rows at a time, over what other rows left in the block."""
    dim, heads = 128, 6
    pool = Pool(nv, 13, heads, dim, [66])
    for i in range(0, 66, rows):
        k = normal(gen(400 + i), rows, heads, dim)
        k[:, 0] = 0.0
        k[:, 1] = 2.0 ** -133
        if i > 30:
            k[0, 1, 3] = -(2.0 ** (i - 130))
            k[:, 2, 1] = torch.finfo(torch.bfloat16).max
            k[0, 3, 5], k[-1, 4, 127] = float("inf"), float("nan")
            k[:, 4, :9] = float("-inf")
        k[:, 5, ::2], k[:, 5, 1::2] = -0.0, 448.0 * 2.0 ** (i // 9)
        v = k.flip(1)
        lens = [i + rows]
        pool.ref.write((k.double().numpy(), v.double().numpy()), [0, rows], lens, pool.table)
        nv.kv_write(pool.gpu, k.cuda(), v.cuda(), i32([0, rows]), i32(lens), pool.tab)
    pool.same()


@pytest.mark.parametrize("fraction", range(128))
def test_power_of_every_fraction(nv, fraction):
    """amax = (1 + f/128) 2^e for every bf16 fraction: the power steps at 1.75, and codes stay at most 448."""
    values = torch.tensor([(1 + fraction / 128) * 2.0 ** e for e in range(-126, 128)], dtype=torch.float64)
    heads = len(values)
    k = torch.zeros(1, heads, 64, dtype=torch.bfloat16)
    k[0, :, 7] = values.to(torch.bfloat16)
    pool = Pool(nv, 1, heads, 64, [1], filled=False)
    nv.kv_write(pool.gpu, k.cuda(), k.cuda(), i32([0, 1]), pool.lens, pool.tab)
    pool.ref.write((k.double().numpy(),) * 2, [0, 1], [1], pool.table)
    pool.same()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("count,rows,past", [(80, 60, 0), (80, 75, 37), (201, 200, 63), (20, 70, 60), (9, 33, 1)])
def test_one_sequence_among_empty_ones(nv, dim, count, rows, past):
    """Many rows of one sequence although there are few rows a sequence: every length of a wave's share."""
    news, pasts = [0] * count, [5] * count
    news[count // 2], pasts[count // 2] = rows, past
    lens = [p + n for p, n in zip(pasts, news)]
    pool = Pool(nv, 500 + rows, 3, dim, lens)
    g = gen(501 + rows)
    k, v = normal(g, rows, 3, dim), normal(g, rows, 3, dim, sigma=30.0)
    rs = starts(news)
    nv.kv_write(pool.gpu, k.cuda(), v.cuda(), i32(rs), pool.lens, pool.tab)
    pool.ref.write((k.double().numpy(), v.double().numpy()), rs, lens, pool.table)
    pool.same()


def test_tokens_appended_one_by_one(nv):
    """150 single appends: each step equals the formula, whatever grew on the way."""
    heads, dim = 3, 128
    pool = Pool(nv, 8, heads, dim, [150])
    g = gen(9)
    k, v = normal(g, 150, heads, dim), normal(g, 150, heads, dim)
    size = torch.exp2(torch.randint(-6, 7, (150, heads, 1), generator=g).float()).to(torch.bfloat16)
    k, v = k * size, v * size.flip(0)
    for i in range(150):
        lens = [i + 1]
        pool.ref.write((k[i:i + 1].double().numpy(), v[i:i + 1].double().numpy()), [0, 1], lens, pool.table)
        nv.kv_write(pool.gpu, k[i:i + 1].cuda(), v[i:i + 1].cuda(), i32([0, 1]), i32(lens), pool.tab)
    pool.same()


@pytest.mark.parametrize("dim,pairs,split", [(64, [32], True), (64, [8], True), (64, [3, 5], False), (128, [16, 24, 24], False),
                                             (128, [22, 21, 21], True), (128, [8, 8], True), (128, [40], True),
                                             (64, [1, 2, 3, 2], True)])
@pytest.mark.parametrize("seqs", [[(0, 130), (37, 1), (60, 70)], [(0, 1), (63, 1), (64, 1)], [(0, 3), (37, 1), (62, 5)]])
def test_kv_write_rotates_the_keys_as_rope_does(nv, dim, pairs, split, seqs):
    heads = 5
    news = [n for _, n in seqs]
    rows = sum(news)
    g = gen(20)
    k, v = normal(g, rows, heads, dim), normal(g, rows, heads, dim)
    size = [9 + a for a in range(len(pairs))]
    tables = [t.cuda() for t in tables_for(pairs, size)]
    positions = torch.stack([torch.randint(0, n, (rows,), generator=g) for n in size], 1).int().cuda()
    one, two = (Pool(nv, 21, heads, dim, [p + n for p, n in seqs]) for _ in range(2))
    rs = i32(starts(news))
    nv.kv_write(one.gpu, strided(k, "qkv"), v.cuda(), rs, one.lens, one.tab, tables=tables, positions=positions, split=split)
    turned = nv.rope(k.cuda(), tables, positions, split=split)
    nv.kv_write(two.gpu, turned, v.cuda(), rs, two.lens, two.tab)
    for a, b in zip(one.pulled(), two.pulled()):
        assert np.array_equal(a, b)


def test_kv_write_and_read_past_the_ends(nv):
    """Rows outside the sequences, more rows than positions, blocks and lengths that do not exist."""
    heads, dim = 2, 64
    k = normal(gen(30), 80, heads, dim)
    pool = Pool(nv, 31, heads, dim, [70, 20, 64, 40, 100])
    pool.table[2, 0] = pool.ref.blocks          # outside the pool
    pool.table[3, 0] = -1
    lens = [70, 20, 64, 40, 4 * BLOCK]          # the last is more than the table holds
    rs = [3, 13, 43, 53, 63, 73]                # rows 0..2 and 73..79 belong to nobody; sequence 1 has 30 rows for 20
    tab = i32(pool.table.tolist())
    pool.ref.write((k.double().numpy(),) * 2, rs, lens, pool.table)
    nv.kv_write(pool.gpu, k.cuda(), k.cuda(), i32(rs), i32(lens), tab)
    pool.same()
    out = [torch.full((80, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    nv.kv_read(pool.gpu, 80, i32(rs), i32(lens), tab, k=out[0], v=out[1])
    for kind in range(2):
        got = out[kind].cpu().double().numpy()
        assert (got[:3] == 5).all() and (got[73:] == 5).all()
        for h in range(heads):
            assert np.array_equal(got[3:13, h], pool.ref.sequence(kind, h, pool.table[0], 70)[60:])
            assert (got[13:23, h] == 0).all()
            assert np.array_equal(got[23:43, h], pool.ref.sequence(kind, h, pool.table[1], 20))
        assert np.isnan(got[43:73]).all()


@BOUNDS
@pytest.mark.parametrize("rs,lens", [([5, 2, 9], [4, 4]), ([-3, 40, 2000], [64, 64]), ([0, 0, 0], [0, 0]),
                                     ([10, 10, 3], [2**31 - 1, -2**31]), ([2**31 - 1, -2**31, 5], [64, -1])])
def test_arrays_that_make_no_sense_stay_in_bounds(nv, rs, lens):
    """Row starts and lengths of any content: no access leaves the arrays (checked by what surrounds them)."""
    heads, dim, M = 2, 64, 12
    k = normal(gen(33), M, heads, dim).cuda()
    pool = Pool(nv, 34, heads, dim, [64, 64])
    tab = pool.tab
    nv.kv_write(pool.gpu, k, k, i32(rs), i32(lens), tab)
    big = torch.full((M + 20, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    nv.kv_read(pool.gpu, M, i32(rs), i32(lens), tab, k=big[10:10 + M], v=torch.empty_like(k))
    assert bool((big[:10] == 5).all()) and bool((big[10 + M:] == 5).all())
    big.fill_(5.0)
    nv.kv_attention(k, pool.gpu, i32(rs), i32(lens), tab, out=big[10:10 + M], causal_block=1)
    assert bool((big[:10] == 5).all()) and bool((big[10 + M:] == 5).all())


@pytest.mark.parametrize("dim,heads,seqs", [(64, 1, [(0, 1)]), (128, 3, [(10, 60), (0, 200)]), (64, 5, [(63, 2), (64, 64), (0, 0)]),
                                            (128, 1, [(500, 77)])])
@pytest.mark.parametrize("layout", ["plain", "qkv", "heads"])
def test_kv_read(nv, dim, heads, seqs, layout):
    news = [n for _, n in seqs]
    lens = [p + n for p, n in seqs]
    pool = Pool(nv, 40 + dim, heads, dim, lens)
    rs, rows = starts(news), sum(news)
    k, v = (strided(torch.zeros(rows, heads, dim, dtype=torch.bfloat16), layout) for _ in range(2))
    got = nv.kv_read(pool.gpu, rows, i32(rs), pool.lens, pool.tab, k=k, v=v)
    assert got[0] is k and got[1] is v
    for b, (past, n) in enumerate(seqs):
        for kind in range(2):
            for h in range(heads):
                want = pool.ref.sequence(kind, h, pool.table[b], past + n)[past:]
                assert np.array_equal(got[kind][rs[b]:rs[b + 1], h].cpu().double().numpy(), want)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def check(got, want, tol):
    got = got.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in other places"
    bad = ~np.isnan(want) & (np.abs(got - want) > tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - want) / tol):.3g} of the bound"


ATTENTION = [
    # dim, kv heads, group, causal block, [(past, new)]
    (64, 1, 1, 0, [(0, 1)]),
    (128, 1, 1, 1, [(0, 1)]),
    (128, 2, 4, 1, [(516, 1)]),
    (64, 3, 1, 1, [(63, 1), (64, 1), (65, 1), (0, 1)]),
    (128, 2, 5, 1, [(300, 1), (0, 1), (77, 1), (900, 1)]),
    (64, 2, 8, 1, [(100, 3), (10, 2), (0, 3), (5, 0)]),
    (128, 1, 1, 1, [(0, 33), (0, 70)]),
    (128, 2, 3, 1, [(0, 65), (17, 100)]),
    (64, 2, 2, 0, [(40, 90), (0, 129)]),
    (128, 1, 4, 16, [(5, 60), (64, 48)]),
    (64, 2, 1, 100, [(0, 250)]),
    (128, 3, 1, 0, [(1, 200)]),
    (64, 1, 40, 1, [(70, 3)]),
    (128, 1, 1, 1, [(3000, 1)]),
]


@BOUNDS
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(nv, case):
    dim, heads, group, c, seqs = ATTENTION[case]
    news = [n for _, n in seqs]
    pool = Pool(nv, 50 + case, heads, dim, [p + n for p, n in seqs])
    q = normal(gen(60 + case), sum(news), heads * group, dim, sigma=1.0 + case % 3)
    rs, scale = starts(news), dim ** -0.5
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, rs, pool.lens.tolist(), pool.table, np.float64(np.float32(scale)),
                                 c, bounds=True)
    for layout in ("plain", "qkv", "heads"):
        got = nv.kv_attention(strided(q, layout), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c)
        check(got, want, tol)
    out = strided(torch.zeros_like(q), "heads")
    nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c, out=out)
    assert same(out, got)
    inplace = q.cuda()
    nv.kv_attention(inplace, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c, out=inplace)
    assert same(inplace, got)


@BOUNDS
@pytest.mark.parametrize("dim,heads,group,c,seqs", [(128, 2, 4, 1, [(0, 700), (333, 500)]), (64, 3, 1, 0, [(900, 601)]),
                                                    (128, 4, 1, 256, [(100, 1100)]), (64, 2, 7, 1, [(0, 300), (0, 301)])])
def test_attention_of_longer_rows(nv, dim, heads, group, c, seqs):
    news = [n for _, n in seqs]
    pool = Pool(nv, 70, heads, dim, [p + n for p, n in seqs])
    q = normal(gen(71), sum(news), heads * group, dim)
    rs, scale = starts(news), np.float64(np.float32(0.1))
    want, tol = kv_ref.attention_fast(q.double().numpy(), pool.ref, rs, pool.lens.tolist(), pool.table, scale, c)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, scale=0.1, causal_block=c)
    check(got, want, tol)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_len", [0, 64, 1000, 2100, 4000, 5000, 12000, 200000])
def test_attention_is_right_for_any_bound_on_the_lengths(nv, max_len, dim):
    """max_len decides the number of parts only (1, 4, 7, 9, 23 and 64 here); below and above the true lengths the
    result stays right."""
    pool = Pool(nv, 80, 2, dim, [2000, 1, 130])
    q = normal(gen(81), 3, 8, dim)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, [0, 1, 2, 3], [2000, 1, 130], pool.table,
                                 np.float64(np.float32(dim ** -0.5)), 1, bounds=True)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32([0, 1, 2, 3]), pool.lens, pool.tab, causal_block=1, max_len=max_len)
    check(got, want, tol)


@pytest.mark.parametrize("dim,count", [(64, 12), (128, 12), (64, 16)])
def test_attention_in_two_parts(nv, dim, count):
    """Many workgroups already: the keys in two parts only, or from 16 sequences on in four."""
    heads = 16
    r = np.random.RandomState(count)
    lens = [2100] + r.randint(1, 2100, count - 1).tolist()
    pool = Pool(nv, 106, heads, dim, lens)
    rs = list(range(count + 1))
    parts = 2 if count < 16 else 4
    assert nv.nvfp4_kv_attention_workspace_bytes(count, count, heads, heads, dim, 2112) == parts * count * heads * (dim + 2) * 4
    q = normal(gen(107), count, heads, dim)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, rs, lens, pool.table, np.float64(np.float32(dim ** -0.5)), 1,
                                 bounds=True)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1)
    check(got, want, tol)


@BOUNDS
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_rows_that_see_nothing(nv, rows):
    """A sequence of no positions, and more rows than positions under a causal mask: those rows are 0, and rows of no
    sequence are left as they were."""
    pool = Pool(nv, 82, 1, 64, [0, 5, 70])
    rs = [2, 2 + rows, 2 + 2 * rows, 2 + 3 * rows]
    q = normal(gen(83), rs[-1] + 3, 2, 64)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1, out=out)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, rs, [0, 5, 70], pool.table, np.float64(np.float32(0.125)), 1,
                                 bounds=True)
    inside = slice(rs[0], rs[-1])
    check(out[inside], want[inside], tol[inside])
    assert bool((out[:rs[0]] == 5).all()) and bool((out[rs[-1]:] == 5).all())
    assert bool((out[rs[0]:rs[1]] == 0).all())
    if rows > 5:
        assert bool((out[rs[1]:rs[2] - 5] == 0).all())


@BOUNDS
@pytest.mark.parametrize("dim,group,news,past", [
    (64, 1, [1, 1], [70, 100]), (128, 2, [40, 3], [70, 100]), (128, 1, [150, 130], [70, 100]), (64, 4, [200, 70], [70, 100]),
    (128, 2, [3, 1], [2500, 3001]), (64, 1, [150, 99], [2500, 1900])])  # the last two share the keys out
def test_what_is_hidden_has_no_effect(nv, dim, group, news, past):
    """NaN codes behind the last position and in masked places: the outputs' bytes do not change.  A NaN that a row
    sees reaches that row, and no other."""
    lens = [p + n for p, n in zip(past, news)]
    pool = Pool(nv, 84, 2, dim, lens)
    q = normal(gen(85), sum(news), 2 * group, dim)
    rs = starts(news)
    call = lambda: nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1)  # noqa: E731
    clean = call()
    for b in range(2):  # the tail of the last block, keys, values
        tail = lens[b] % BLOCK
        page = pool.table[b, lens[b] // BLOCK] if tail else None
        if page is not None:
            for kind in range(2):
                pool.ref.codes[kind][page][:, pool.ref.off[kind][tail:]] = 0x7F
    pool.push()
    assert same(call(), clean)
    # one NaN in head 1 of sequence 0, at a position that only some rows see
    at = past[0] + news[0] // 2
    for kind in range(2):
        pool.ref.codes[kind][pool.table[0, at // BLOCK], 1, pool.ref.off[kind][at % BLOCK, 3]] = 0xFF
        pool.push()
        got, nan = call().cpu(), torch.zeros(q.shape, dtype=torch.bool)
        i = torch.arange(news[0])[past[0] + torch.arange(news[0]) >= at]
        if kind == 0:
            nan[i, group:] = True
        else:
            nan[i, group:, 3] = True
        assert torch.equal(got.isnan(), nan)
        assert np.array_equal(bits(got)[~nan.numpy()], bits(clean)[~nan.numpy()])
        pool.ref.codes[kind][pool.table[0, at // BLOCK], 1, pool.ref.off[kind][at % BLOCK, 3]] = 0x30
        pool.push()
        clean = call()


@BOUNDS
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 1), (64, 3), (128, 5), (64, 66), (128, 130), (64, 201)])
def test_codes_left_behind_the_largest_values(nv, dim, rows, causal):
    """A block whose values need the largest power, 2^120, with the codes of an earlier use (448, which times 2^120
    is not finite) behind the last position: they have no effect.  Zero keys, so all probabilities are 1 before the
    division; the largest value is the only one of its block that is not rounded to 0, so every sum is finite."""
    v = torch.ones(rows, 2, dim, dtype=torch.bfloat16)
    v[-1, 0, 3] = torch.finfo(torch.bfloat16).max
    v[-1, 1, dim - 1] = -torch.finfo(torch.bfloat16).max
    q = normal(gen(dim + rows), rows, 4, dim)
    blocks = -(-rows // BLOCK)
    got = []
    for left in (0, 0x7E):
        cache = nv.KvCache.empty(blocks, 2, dim)
        for t in (cache.k, cache.v):
            t.fill_(left)
        args = i32([0, rows]), i32([rows]), i32([list(range(blocks))])
        nv.kv_write(cache, torch.zeros_like(v).cuda(), v.cuda(), *args)
        got.append(nv.kv_attention(q.cuda(), cache, *args, causal_block=causal))
    assert bool(torch.isfinite(got[0]).all()) and bool((got[0][-1, :2, 3] > 2.0 ** 110).all())
    assert same(got[1], got[0])


@BOUNDS
@pytest.mark.parametrize("rows", [1, 50, 200])
def test_blocks_and_lengths_that_do_not_exist(nv, rows):
    pool = Pool(nv, 86, 2, 64, [300, 300, 300, 300])
    pool.table[1, 1] = pool.ref.blocks
    pool.table[2, 4] = -2
    lens = [300, 300, 300, 6 * BLOCK]
    rs = [0, rows, 2 * rows, 3 * rows, 4 * rows]
    q = normal(gen(87), 4 * rows, 2, 64)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32(rs), i32(lens), i32(pool.table.tolist()), causal_block=1)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, rs, lens, pool.table, np.float64(np.float32(0.125)), 1, bounds=True)
    check(got, want, tol)
    assert np.isnan(want[3 * rows:]).all() and not np.isnan(want[:rows]).any()


@BOUNDS
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [30, 130])
def test_missing_blocks_beside_unwritten_ones(nv, dim, rows):
    """Rows that do not see a missing block, in a tile whose other rows do: they are what they are without it, also
    where the pool's first block, never written, holds what is not finite."""
    past = 40  # the first 24 rows end before the missing block 1
    n = past + rows
    blocks = -(-n // BLOCK)
    k, v, q = (normal(gen(700 + i), *s) for i, s in enumerate(((n, 2, dim), (n, 2, dim), (rows, 2, dim))))
    table = [list(range(1, blocks + 1))]
    cache = nv.KvCache.empty(blocks + 1, 2, dim)
    nv.kv_write(cache, k.cuda(), v.cuda(), i32([0, n]), i32([n]), i32(table))
    table[0][1] = -1
    got = []
    for code, power in ((0, 1), (0x7E, 254), (0x7F, 255)):
        for t, x in ((cache.k, code), (cache.v, code), (cache.k_power, power), (cache.v_power, power)):
            t[0] = x
        got.append(nv.kv_attention(q.cuda(), cache, i32([0, rows]), i32([n]), i32(table), causal_block=1))
    for x in got:
        assert bool(torch.isfinite(x[:24]).all()) and bool(x[24:].isnan().all())
        assert same(x[:24], got[0][:24])


@BOUNDS
def test_queries_that_are_not_finite_and_large_and_small_ones(nv):
    pool = Pool(nv, 88, 1, 128, [100, 100])
    q = normal(gen(89), 40, 1, 128)
    q[3, 0, 5], q[20, 0, 100], q[21, 0, 0] = float("nan"), float("inf"), float("-inf")
    q[4] = 0.0
    q[5] *= 2.0 ** -100
    q[6] = 2.0 ** -133
    q[7] *= 16.0
    q[8, 0, ::2] *= 2.0 ** -14
    rs = [0, 20, 40]
    got = nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1)
    clean = q.double().numpy().copy()
    bad = ~np.isfinite(clean).all(axis=2)
    clean[bad] = 0.0
    want, tol = kv_ref.attention(clean, pool.ref, rs, [100, 100], pool.table, np.float64(np.float32(128 ** -0.5)), 1, bounds=True)
    want[bad] = np.nan
    check(got, want, tol)


@BOUNDS
def test_values_of_very_different_powers(nv):
    """Blocks whose values differ by powers of two up to 2^60, and values near the ends of the range."""
    for low, high in ((90, 150), (10, 30), (200, 240)):
        pool = Pool(nv, 90, 2, 128, [640])
        r = np.random.RandomState(91)
        pool.ref.powers[1][:] = r.randint(low, high, pool.ref.powers[1].shape)
        pool.push()
        q = normal(gen(92), 50, 2, 128)
        got = nv.kv_attention(q.cuda(), pool.gpu, i32([0, 50]), pool.lens, pool.tab, causal_block=1)
        want, tol = kv_ref.attention_fast(q.double().numpy(), pool.ref, [0, 50], [640], pool.table,
                                          np.float64(np.float32(128 ** -0.5)), 1)
        check(got, want, tol)


@BOUNDS
def test_scores_far_apart(nv):
    """A growing row of scores (each block above the last by hundreds), a falling one, and one that stays."""
    heads, dim, n = 3, 64, 640
    pool = Pool(nv, 93, heads, dim, [n])
    pool.ref.codes[0][:] = 0x38  # 1.0
    for at in range(10):
        page = pool.table[0, at]
        pool.ref.powers[0][page, 0] = 127 + at - 6
        pool.ref.powers[0][page, 1] = 127 + 3 - at
        pool.ref.powers[0][page, 2] = 127
    pool.push()
    q = torch.ones(5, heads, dim, dtype=torch.bfloat16) * torch.tensor([1.0, -1.0, 0.1, 3.0, 40.0])[:, None, None].to(torch.bfloat16)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32([0, 5]), pool.lens, pool.tab, scale=1.0)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, [0, 5], [n], pool.table, 1.0, 0, bounds=True)
    check(got, want, tol)


@BOUNDS
@pytest.mark.parametrize("count", [62, 63, 64, 65, 300, 4200])
def test_many_sequences(nv, count):
    """Counts around and above the 64 that are looked up at once: written, read back and attended, each sequence by
    itself; some have no rows."""
    heads, dim = 1, 64
    g = gen(count)
    news = torch.randint(0, 4, (count,), generator=g).tolist()
    past = torch.randint(0, 70, (count,), generator=g).tolist()
    lens = [p + n for p, n in zip(past, news)]
    pool = Pool(nv, count, heads, dim, lens)
    rows, rs = sum(news), starts(news)
    k, v, q = (normal(g, rows, n, dim) for n in (heads, heads, 2))
    nv.kv_write(pool.gpu, k.cuda(), v.cuda(), i32(rs), pool.lens, pool.tab)
    pool.ref.write((k.double().numpy(), v.double().numpy()), rs, lens, pool.table)
    pool.same()
    back = nv.kv_read(pool.gpu, rows, i32(rs), pool.lens, pool.tab)
    want = [np.concatenate([pool.ref.sequence(kind, 0, pool.table[b], lens[b])[past[b]:] for b in range(count)]) for kind in range(2)]
    for kind in range(2):
        assert np.array_equal(back[kind][:, 0].cpu().double().numpy(), want[kind])
    got = nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1)
    ref, tol = kv_ref.attention(q.double().numpy(), pool.ref, rs, lens, pool.table, np.float64(np.float32(0.125)), 1, bounds=True)
    check(got, ref, tol)


@BOUNDS
@pytest.mark.parametrize("count,rows,group,dim,longest", [
    (70, {0: 1}, 1, 64, 2500), (70, {69: 1}, 4, 128, 2500), (300, {3: 1, 150: 2, 151: 1, 299: 1}, 2, 64, 1500),
    (9, {2: 1, 7: 1}, 40, 64, 2500), (12, {0: 1, 5: 2}, 70, 128, 600), (12, {1: 1, 2: 1, 11: 1}, 130, 64, 1100),
    (8, {b: 1 for b in range(8)}, 300, 64, 700), (64, {b: 1 for b in range(64)}, 3, 64, 300), (40, {9: 35}, 3, 64, 900)])
def test_slots_that_are_mostly_empty(nv, count, rows, group, dim, longest):
    """A few sequences with rows among many without, one to several tiles a row, rows before the first sequence and
    after the last: written, read back and attended."""
    g = gen(count + group)
    news = [rows.get(b, 0) for b in range(count)]
    lens = [int(torch.randint(news[b], longest if news[b] else 60, (1,), generator=g)) for b in range(count)]
    lens[max(rows)] = longest
    pool = Pool(nv, count + dim, 1, dim, lens)
    lead, n = 2, sum(news)
    M, rs = lead + n + 3, [lead + r for r in starts(news)]
    k, v, q = (normal(g, M, h, dim) for h in (1, 1, group))
    nv.kv_write(pool.gpu, k.cuda(), v.cuda(), i32(rs), pool.lens, pool.tab)
    pool.ref.write((k.double().numpy(), v.double().numpy()), rs, lens, pool.table)
    pool.same()
    out = [torch.full((M, h, dim), 5.0, dtype=torch.bfloat16, device="cuda") for h in (1, 1, group)]
    nv.kv_read(pool.gpu, M, i32(rs), pool.lens, pool.tab, k=out[0], v=out[1])
    nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1, out=out[2])
    for x in out:
        assert bool((x[:lead] == 5).all()) and bool((x[lead + n:] == 5).all())
    for kind in range(2):
        want = np.concatenate([pool.ref.sequence(kind, 0, pool.table[b], lens[b])[lens[b] - news[b]:] for b in range(count)])
        assert np.array_equal(out[kind][lead:lead + n, 0].cpu().double().numpy(), want)
    mid = slice(lead, lead + n)
    want, tol = kv_ref.attention(q[mid].double().numpy(), pool.ref, starts(news), lens, pool.table,
                                 np.float64(np.float32(dim ** -0.5)), 1, bounds=True)
    check(out[2][mid], want, tol)


@BOUNDS
def test_sequences_that_share_blocks(nv):
    """A prefix's blocks in several tables, and a block twice in one: read only, each sequence as if alone."""
    pool = Pool(nv, 108, 2, 64, [300, 300, 300])
    pool.table[1, :3] = pool.table[0, :3]
    pool.table[2] = pool.table[2, 0]
    lens, rs = [300, 250, 300], [0, 1, 41, 241]
    q = normal(gen(109), 241, 4, 64)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, rs, lens, pool.table, np.float64(np.float32(0.125)), 1, bounds=True)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32(rs), i32(lens), i32(pool.table.tolist()), causal_block=1)
    check(got, want, tol)


def test_a_pool_past_4_gib(nv):
    """Blocks whose offsets pass 32 bits: the same rows through the pool's first and last blocks."""
    heads, dim, n = 8, 128, 200
    blocks = 2**32 // (heads * 64 * dim) + 100  # 4 GiB of keys and as much of values
    pool = nv.KvCache.empty(blocks, heads, dim)
    g = gen(7)
    k, v, q = (normal(g, n, h, dim).cuda() for h in (heads, heads, 2 * heads))
    rs, lens = i32([0, n]), i32([n])
    got = []
    for table in ([0, 1, 2, 3], [blocks - 1, blocks - 90, blocks - 2, blocks - 50]):
        tab = i32([table])
        nv.kv_write(pool, k, v, rs, lens, tab)
        got.append([*nv.kv_read(pool, n, rs, lens, tab), nv.kv_attention(q, pool, rs, lens, tab, causal_block=1),
                    nv.kv_attention(q[-1:], pool, i32([0, 1]), lens, tab, causal_block=1)])
    for a, b in zip(*got):
        assert same(a, b)
    assert float(got[0][0].double().abs().max()) > 1


def test_rows_further_apart_than_2_gib(nv):
    """Row strides of 2^31 elements: inputs and outputs of each operator spread over one allocation."""
    heads, dim, stride = 2, 64, 2**31
    store = torch.zeros(2 * stride + heads * dim, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(store, (3, heads, dim), (stride, dim, 1))
    g = gen(8)
    x = normal(g, 3, heads, dim).cuda()
    tables = [nv.rope_table(9, 16)]
    pos = i32([[1], [8], [0]])
    near = nv.rope(x, tables, pos)
    far.copy_(x)
    assert same(nv.rope(far, tables, pos), near)
    nv.rope(far, tables, pos, out=far)
    assert same(far, near)
    one, two = (Pool(nv, 9, heads, dim, [3], filled=False) for _ in range(2))
    rs = i32([0, 3])
    nv.kv_write(one.gpu, near, near, rs, one.lens, one.tab)
    nv.kv_write(two.gpu, far, far, rs, two.lens, two.tab)
    for a, b in zip(one.pulled(), two.pulled()):
        assert np.array_equal(a, b)
    want = nv.kv_attention(near, one.gpu, rs, one.lens, one.tab)
    assert same(nv.kv_attention(far, one.gpu, rs, one.lens, one.tab), want)
    back = nv.kv_read(one.gpu, 3, rs, one.lens, one.tab)
    nv.kv_attention(near, one.gpu, rs, one.lens, one.tab, out=far)
    assert same(far, want)
    nv.kv_read(one.gpu, 3, rs, one.lens, one.tab, k=far, v=torch.empty_like(near))
    assert same(far, back[0])


# ---------------------------------------------------------------------------
# streams, graphs, and the whole run
# ---------------------------------------------------------------------------
def _serving_state(nv, seed, lens, heads=2, group=4, dim=128):
    pool = Pool(nv, seed, heads, dim, [n + 8 for n in lens], filled=False)
    g = gen(seed)
    past = torch.randn(sum(lens), heads, dim, generator=g).to(torch.bfloat16).cuda()
    nv.kv_write(pool.gpu, past, past.flip(0), i32(starts(lens)), i32(lens), pool.tab)
    return pool


@BOUNDS
def test_captured_tokens_replay(nv):
    """Append and attend for four sequences captured once and replayed with new inputs and lengths, eager work in
    between, two graphs alive at once: every replay equals the eager calls."""
    lens = [70, 1, 600, 127]
    one, two = _serving_state(nv, 95, lens), _serving_state(nv, 95, lens)
    third = _serving_state(nv, 95, lens)
    tables = [nv.rope_table(1024, 64)]
    g = gen(96)
    new = lambda: torch.randn(4, 16, 128, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    rs = i32([0, 1, 2, 3, 4])

    def step(pool, x, n, pos):
        q = nv.rope(x[:, :8], tables, pos)
        nv.kv_write(pool.gpu, x[:, 8:10], x[:, 10:12], rs, n, pool.tab, tables=tables, positions=pos)
        return nv.kv_attention(q, pool.gpu, rs, n, pool.tab, causal_block=1)

    made = []
    for pool in (one, two):
        x, n, pos = new(), i32(lens), i32([[p] for p in lens])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(pool, x, n, pos)
        made.append((graph, x, n, pos, out))
    for i in range(6):
        x = new()
        now = [p + i + 1 for p in lens]
        want = step(third, x, i32(now), i32([[p - 1] for p in now])).clone()
        for graph, gx, gn, gpos, out in made:
            gx.copy_(x), gn.copy_(i32(now)), gpos.copy_(i32([[p - 1] for p in now]))
            graph.replay()
        torch.cuda.synchronize()
        for pool, (_, _, _, _, out) in zip((one, two), made):
            assert same(out, want), f"replay {i}"
            for a, b in zip(pool.pulled(), third.pulled()):
                assert np.array_equal(a, b)


def test_other_streams(nv):
    """Calls on side streams, two at once with workspaces of their own, equal the calls on the main one."""
    pool = Pool(nv, 97, 2, 128, [3000])
    q = normal(gen(98), 1, 8, 128).cuda()
    rs = i32([0, 1])
    want = nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in side:
            got.append(nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab, stream=s))
    for s in side:
        s.synchronize()
    for o in got:
        assert same(o, want)


@BOUNDS
def test_same_call_same_bytes(nv):
    pool = Pool(nv, 99, 4, 64, [5000, 4000])
    q = normal(gen(98), 300, 8, 64).cuda()
    for rs in ([0, 1, 2], [0, 150, 300]):
        rows = rs[-1]
        runs = [bits(nv.kv_attention(q[:rows], pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1)) for _ in range(4)]
        assert all(np.array_equal(runs[0], r) for r in runs[1:])


def test_from_projection_to_projection(nv):
    """The run as it is used: modulation producer, QKV product, rotation, cache, attention, plain quantizer, output
    product, for a prompt and then single tokens; attention's inputs and outputs checked against the references."""
    heads, dim, width = 2, 128, 512
    g = gen(101)
    w_qkv = nv.quantize_weight(normal(g, 3 * heads * dim, width, sigma=width ** -0.5).cuda())
    w_out = nv.quantize_weight(normal(g, width, heads * dim, sigma=0.06).cuda())
    shift, scale = normal(g, 1, width, sigma=0.1).cuda(), normal(g, 1, width, sigma=0.1).cuda()
    tables = [nv.rope_table(64, p) for p in (16, 24, 24)]
    pool = Pool(nv, 102, heads, dim, [200], filled=False)
    length = 0
    for rows in (150, 1, 1, 40):
        x = normal(g, rows, width).cuda()
        q8, sf, ts, _ = nv.modulate_quantize(x, [0, rows], shift, scale)
        qkv = nv.gemm(q8, sf, ts, rows, *w_qkv).view(rows, 3 * heads, dim)
        at = torch.arange(length, length + rows)
        positions = torch.stack([at // 24, at // 6 % 4, at % 6], 1).int().cuda()
        length += rows
        rs, lens = i32([0, rows]), i32([length])
        q = nv.rope(qkv[:, :heads], tables, positions)
        nv.kv_write(pool.gpu, qkv[:, heads:2 * heads], qkv[:, 2 * heads:], rs, lens, pool.tab, tables=tables,
                    positions=positions)
        o = nv.kv_attention(q, pool.gpu, rs, lens, pool.tab, causal_block=1)
        host = qkv.cpu()
        cpu_tables = [t.cpu() for t in tables]
        turned = [kv_ref.rotate(host[:, w:w + heads], cpu_tables, positions.cpu(), False).to(torch.bfloat16).double().numpy()
                  for w in (0, heads)]
        pool.ref.write((turned[1], host[:, 2 * heads:].double().numpy()), [0, rows], [length], pool.table)
        pool.same()
        want, tol = kv_ref.attention(turned[0], pool.ref, [0, rows], [length], pool.table,
                                     np.float64(np.float32(dim ** -0.5)), 1, bounds=True)
        check(o, want, tol)
        o8, of, ot, _ = nv.quantize(o.reshape(rows, heads * dim))
        y = nv.gemm(o8, of, ot, rows, *w_out)
        assert tuple(y.shape) == (rows, width) and bool(y.isfinite().all())


def test_c_entry_points_by_name(nv):
    """The functions named like the C entry points, on the structures that the conveniences build, with a workspace of
    the caller's: the same bytes."""
    heads, dim, n = 2, 64, 3000
    g = gen(104)
    k, v, q = (normal(g, n, h, dim).cuda() for h in (heads, heads, 4))
    dev = k.device
    one, two = (Pool(nv, 105, heads, dim, [n], filled=False) for _ in range(2))
    table = torch.empty(50, 32, 2, device="cuda")
    nv.nvfp4_rope_table(table, 50, 32, 10000.0)
    assert torch.equal(table, nv.rope_table(50, 32))
    pos = (torch.arange(n).int() % 50)[:, None].cuda()
    rs, lens = i32([0, n]), i32([n])
    r, s = nv.make_rope_params([table], pos, n, True, dev), nv.make_kv_sequences(rs, lens, two.tab, dev)
    turned = nv.rope(q, [table], pos, split=True)
    out = torch.empty_like(q)
    nv.nvfp4_rope(nv.make_heads("q", q), n, 4, dim, r, nv.make_heads("out", out))
    assert same(out, turned)
    nv.kv_write(one.gpu, k, v, rs, lens, one.tab, tables=[table], positions=pos, split=True)
    nv.nvfp4_kv_write(two.gpu.struct, s, n, nv.make_heads("k", k), nv.make_heads("v", v), r)
    for a, b in zip(one.pulled(), two.pulled()):
        assert np.array_equal(a, b)
    back = torch.empty_like(k), torch.empty_like(v)
    nv.nvfp4_kv_read(two.gpu.struct, s, n, nv.make_heads("k", back[0]), nv.make_heads("v", back[1]))
    for a, b in zip(back, nv.kv_read(one.gpu, n, rs, lens, one.tab)):
        assert same(a, b)
    last = i32([0, 1])
    want = nv.kv_attention(turned[-1:], one.gpu, last, lens, one.tab)
    need = nv.nvfp4_kv_attention_workspace_bytes(1, 1, 4, heads, dim, 64 * one.table.shape[1])
    assert need > 0
    ws, got = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
    s1 = nv.make_kv_sequences(last, lens, two.tab, dev)
    nv.nvfp4_kv_attention(nv.make_heads("q", turned[-1:]), 1, 4, two.gpu.struct, s1, dim ** -0.5, 0, 64 * one.table.shape[1],
                          nv.make_heads("out", got), ws, need)
    assert same(got, want)
    assert same(nv.kv_attention(turned[-1:], one.gpu, last, lens, one.tab, workspace=ws), want)
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_attention(turned[-1:], one.gpu, last, lens, one.tab, workspace=ws[:need // 2])


def test_another_devices_or_types_are_refused(nv):
    pool = Pool(nv, 103, 1, 64, [64])
    q = normal(gen(1), 4, 1, 64)
    rs = i32([0, 4])
    with pytest.raises(ValueError):
        nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab)
    with pytest.raises(ValueError):
        nv.kv_attention(q.cuda(), pool.gpu, rs.cpu(), pool.lens, pool.tab)
    with pytest.raises(TypeError):
        nv.kv_attention(q.cuda().float(), pool.gpu, rs, pool.lens, pool.tab)
    with pytest.raises(TypeError):
        nv.kv_attention(q.cuda(), pool.gpu, rs.long(), pool.lens, pool.tab)
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_attention(q.cuda(), pool.gpu, rs, pool.lens, pool.tab, scale=0.0)
    for c in (-1, 2**31, 2**32):
        with pytest.raises(ValueError):
            nv.kv_attention(q.cuda(), pool.gpu, rs, pool.lens, pool.tab, causal_block=c)
    with pytest.raises(ValueError):
        nv.rope_table(4, 2**32 + 8)
    with pytest.raises(nv.Nvfp4Error):  # an output whose heads overlap
        nv.kv_attention(q.cuda(), pool.gpu, rs, pool.lens, pool.tab, out=torch.empty_like(q.cuda()[:1]).expand(4, 1, 64))
    with pytest.raises(ValueError):
        nv.kv_write(pool.gpu, q.cuda(), q.cuda()[:3], rs, pool.lens, pool.tab)
    with pytest.raises(ValueError):
        nv.kv_write(pool.gpu, q.cuda(), q.cuda(), rs, pool.lens, pool.tab, tables=[nv.rope_table(4, 8)])
    with pytest.raises(nv.Nvfp4Error):  # 4 pairs
        nv.rope(q.cuda(), [nv.rope_table(4, 4)], torch.zeros(4, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(nv.Nvfp4Error):  # positions without a row of their own
        nv.rope(q.cuda(), [nv.rope_table(4, 8)], torch.zeros(1, 1, dtype=torch.int32, device="cuda").expand(4, 1))
    empty = nv.kv_attention(q.cuda()[:0], pool.gpu, i32([0, 0]), pool.lens, pool.tab)
    assert tuple(empty.shape) == (0, 1, 64)


@BOUNDS
@pytest.mark.parametrize("rows", [1, 90])
def test_the_smallest_scale(nv, rows):
    """The smallest number of binary32, not a normal one: all scores are equal, and what is masked stays so."""
    pool = Pool(nv, 110, 2, 64, [200])
    q = normal(gen(111), rows, 4, 64)
    got = nv.kv_attention(q.cuda(), pool.gpu, i32([0, rows]), pool.lens, pool.tab, scale=1e-45, causal_block=1)
    want, tol = kv_ref.attention(q.double().numpy(), pool.ref, [0, rows], [200], pool.table, np.float64(np.float32(1e-45)), 1,
                                 bounds=True)
    check(got, want, tol)


@pytest.mark.parametrize("rope", ["none", "pairs", "split"])
@pytest.mark.parametrize("case", range(len(kv_ref.HEAD_LOOPS)))
def test_several_heads_to_a_workgroup(nv, case, rope):
    """Long writes and reads whose workgroups go over several heads, the last of them over fewer, equal the same rows
    one head at a time: partial first and last blocks over what is there, powers that grow, and rows that are not
    finite in neighbouring heads, in single ones and in none."""
    heads, dim, seqs, _, _ = kv_ref.HEAD_LOOPS[case]
    news, lens = [n for _, n in seqs], [p + n for p, n in seqs]
    M, rs = sum(news), i32(starts(news))
    g = torch.Generator("cuda")
    g.manual_seed(case)
    k, v = (torch.randn(M, heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for x in (k, v):  # sizes of their own for heads and stretches of rows
        x *= torch.exp2(torch.randint(-6, 7, (M // 50 + 1, heads, 1), generator=g, device="cuda")
                        .repeat_interleave(50, 0)[:M].float()).to(torch.bfloat16)
    for h, first, step in ((1, 3, 401), (2, 5, 401), (3, 0, 1009), (7, M - 1, 1), (heads - 1, 2, 333)):
        k[first::step, h, h % dim] = float("inf")
        v[first + 1::step, h, 5] = float("nan")
        v[first::step, h + 1 if h + 1 < heads else 0, 9] = torch.finfo(torch.bfloat16).max
    rot = {}
    if rope != "none":
        pairs = [16, 8, 8] if dim == 64 else [24, 16]
        rot = dict(tables=[t.cuda() for t in tables_for(pairs, [50] * len(pairs))], split=rope == "split",
                   positions=torch.randint(0, 50, (M, len(pairs)), generator=g, device="cuda", dtype=torch.int32))
    need = [-(-n // BLOCK) for n in lens]
    blocks = sum(need) + 1
    order = torch.randperm(blocks, generator=g, device="cuda").int()
    tab = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        tab[b, :n] = order[at:at + n]
        at += n
    pool = nv.KvCache.empty(blocks, heads, dim)
    for t in (pool.k, pool.v):
        t.copy_(torch.randint(0, 0x7F, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (pool.k_power, pool.v_power):
        t.copy_(torch.randint(118, 126, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    ones = [nv.KvCache(*(t[:, h:h + 1].contiguous() for t in (pool.k, pool.v, pool.k_power, pool.v_power))) for h in range(heads)]
    nv.kv_write(pool, k, v, rs, i32(lens), tab, **rot)
    back = nv.kv_read(pool, M, rs, i32(lens), tab)
    for h, one in enumerate(ones):
        nv.kv_write(one, k[:, h:h + 1].contiguous(), v[:, h:h + 1].contiguous(), rs, i32(lens), tab, **rot)
        for name in ("k", "v", "k_power", "v_power"):
            assert torch.equal(getattr(pool, name)[:, h], getattr(one, name)[:, 0]), f"head {h}: {name}"
        for got, want in zip(back, nv.kv_read(one, M, rs, i32(lens), tab)):
            assert torch.equal(got[:, h].view(torch.int16), want[:, 0].view(torch.int16)), f"head {h}"
    bad = torch.isnan(back[1]).any(0).any(1)
    assert bool(bad[1]) and bool(bad[2]) and not bool(bad[10])


@BOUNDS
@pytest.mark.parametrize("dim,heads,group,c,seqs", kv_ref.WIDE_HEADS)
def test_attention_with_heads_for_every_xcd(nv, dim, heads, group, c, seqs):
    """Key/value heads in multiples of 8, which 128-row tiles are laid out by: every row of every head, with odd and
    even numbers of tiles, and no row but those."""
    news = [n for _, n in seqs]
    lens = [p + n for p, n in seqs]
    pool = Pool(nv, 120 + heads, heads, dim, lens)
    lead, n = kv_ref.WIDE_LEAD, sum(news)
    M, rs = n + 2 * lead, [lead + r for r in starts(news)]
    q = normal(gen(121), M, heads * group, dim)
    scale = np.float64(np.float32(dim ** -0.5))
    want, tol = kv_ref.attention_fast(q.double().numpy(), pool.ref, rs, lens, pool.table, scale, c)
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    nv.kv_attention(q.cuda(), pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c, out=out)
    assert bool((out[:lead] == 77).all()) and bool((out[lead + n:] == 77).all())
    check(out[lead:lead + n], want[lead:lead + n], tol[lead:lead + n])


@BOUNDS
@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 1), (64, 40), (128, 200)])
def test_scores_and_values_at_their_documented_ends(nv, dim, rows):
    """Scaled scores up to 2^26, where the reference is off by up to 4 in the exponent, and values up to 2^96: each row
    sees the mean of one block's values, all others being too far below.

    Those 64 probabilities are equal, so their rounding to bf16 (half a step, 2^-8) is one factor of the products that
    their sum does not have; the output's is 2^-8 more, and the sums of 64 terms and the division some 2^-24 each."""
    blocks, heads = 6, 2
    pool = Pool(nv, 130 + dim, heads, dim, [blocks * BLOCK])
    pool.ref.codes[0][:] = 0x38  # 1.0
    pool.ref.powers[1][:] = 127 + 87  # up to 448 * 2^87 < 2^96
    top = (4, 2)
    for h in range(heads):
        for at in range(blocks):
            pool.ref.powers[0][pool.table[0, at], h] = 127 + (10 if at == top[h] else at)
    pool.push()
    # the largest score is dim * 2^20, and scaled 0.61 * 2^26
    q = torch.full((rows, heads, dim), 2.0 ** 10, dtype=torch.bfloat16)
    scale = np.float32(0.61 * 2.0 ** 26 / (dim * 2.0 ** 20))
    got = nv.kv_attention(q.cuda(), pool.gpu, i32([0, rows]), pool.lens, pool.tab, scale=float(scale)).cpu().double().numpy()
    for h in range(heads):
        v = pool.ref.sequence(1, h, pool.table[0], blocks * BLOCK)[top[h] * BLOCK:(top[h] + 1) * BLOCK]
        want, a = v.mean(0), np.abs(v).mean(0)
        off = (2.0 ** -8 + 128 * 2.0 ** -24) * a
        assert (np.abs(got[:, h] - want) <= off + 2.0 ** -8 * (np.abs(want) + off)).all()
