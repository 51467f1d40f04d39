"""Attention through a window and over a shared prefix where the keys are cut into pieces that are joined, and on streams
whose inputs are still being made, against plain references (tests/step_ref.py)."""
import functools

import numpy as np
import pytest
import torch

from tests import kv_ref, step_ref
from tests.gpu_util import device
from tests.test_gpu_attention import Pool, check, gen, i32, normal, same, starts
from tests.test_gpu_step import BOUND, shared_pool, test_what_a_window_hides_has_no_effect as check_hidden

pytestmark = pytest.mark.gpu
BLOCK = 64


@pytest.fixture(scope="module")
def nv():
    import nvfp4_activation_quantization_segment_amd as m

    device()
    return m


def one_dim_a_block(pool, table):
    """Keeps of the values of each sequence's block `at` only dim `at` mod dim, as magnitudes: that output is the weight of
    few blocks (of one, where there are at most dim of them), so that a block left out or taken twice is an error of the
    size of the output itself, and the bound is a few steps of it."""
    dim = pool.dim
    for row in table:
        for at, page in enumerate(row):
            if 0 <= page < pool.ref.blocks:
                kept = np.zeros(BLOCK * dim, bool)
                kept[pool.ref.off[1][:, at % dim]] = True
                codes = pool.ref.codes[1][page]
                codes[:] = np.where(kept, codes & 0x7F, 0)
    pool.push()


def scale_of(dim):
    return np.float64(np.float32(dim ** -0.5))


def window_pieces(nv, rows, count, heads, group, dim, c, window, sinks, max_len):
    need = nv.nvfp4_kv_attention_window_workspace_bytes(rows, count, heads * group, heads, dim, c, window, sinks, max_len)
    return need // (rows * heads * group * (dim + 2) * 4)


# ---------------------------------------------------------------------------
# windows
# ---------------------------------------------------------------------------
PIECES = [
    # dim, kv heads, group, causal block, window, sinks, [(past, new)]
    (128, 2, 4, 1, 4000, 4, [(9000, 1)]),
    (128, 1, 4, 1, 4096, 0, [(4095, 1), (4096, 1), (4097, 1)]),
    (64, 2, 4, 1, 4000, 130, [(9000, 1), (5000, 2), (100, 1), (4200, 1)]),
    (128, 1, 8, 1, 2000, 0, [(7000, 3), (0, 1), (2100, 4)]),
    (64, 1, 3, 1, 2047, 130, [(4097, 1), (2048, 1), (2047, 0), (129, 1), (2200, 3), (6000, 1), (2111, 1)]),
    (128, 2, 1, 16, 2500, 4, [(3000, 5), (2600, 2)]),
    (128, 1, 1, 1, 9000, 130, [(12000, 150)]),          # 128-row tiles
    (64, 2, 2, 1, 8500, 0, [(100, 70), (11000, 80)]),
    (64, 1, 1, 64, 9000, 4, [(9500, 200)]),
]


@functools.lru_cache(maxsize=1)
def window_case(nv, case):
    dim, heads, group, c, window, sinks, seqs = PIECES[case]
    news = [n for _, n in seqs]
    pool = Pool(nv, 400 + case, heads, dim, [p + n for p, n in seqs])
    one_dim_a_block(pool, pool.table)
    q = normal(gen(410 + case), sum(news), heads * group, dim)
    rs = starts(news)
    want = step_ref.attention(q.double().numpy(), pool.ref, rs, pool.lens.tolist(), pool.table, scale_of(dim), c, window, sinks)
    return pool, q.cuda(), rs, want


@pytest.mark.parametrize("case", range(len(PIECES)))
@BOUND
def test_a_window_in_pieces(nv, case, bound):
    """Windows that hide keys, their blocks shared out over workgroups: pieces that hold the first positions and the
    window's beginning, pieces without a key of a shorter sequence, and their join."""
    dim, heads, group, c, window, sinks, seqs = PIECES[case]
    pool, q, rs, (want, tol) = window_case(nv, case)
    most = pool.tab.shape[1] * BLOCK if bound is None else bound
    pieces = window_pieces(nv, len(q), len(seqs), heads, group, dim, c, window, sinks, most)
    assert pieces > 1 if bound != 0 else pieces == 0
    call = lambda: nv.kv_attention(q, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=c, max_len=bound,  # noqa: E731
                                   window=window, sinks=sinks)
    got = call()
    check(got, want, tol)
    assert same(call(), got)


@pytest.mark.parametrize("dim,group,rows,past,window,sinks", [(128, 2, 3, 6000, 4000, 130), (64, 4, 1, 5000, 2100, 4),
                                                              (64, 1, 150, 10000, 8600, 65)])
def test_what_a_window_in_pieces_hides_has_no_effect(nv, dim, group, rows, past, window, sinks):
    assert window_pieces(nv, rows, 1, 2, group, dim, 1, window, sinks, past + rows + BLOCK) > 1
    check_hidden(nv, None, dim, group, rows, past, window, sinks)


# ---------------------------------------------------------------------------
# shared prefixes
# ---------------------------------------------------------------------------
def shared_pieces(nv, rows, count, heads, group, dim, blocks, max_len):
    need = nv.nvfp4_kv_attention_shared_workspace_bytes(rows, count, heads * group, heads, dim, blocks, max_len)
    return need // (rows * heads * group * (dim + 2) * 4)


def check_shared(nv, pool, common, q, rs, bound, want):
    got = nv.kv_attention(q, pool.gpu, i32(rs), pool.lens, pool.tab, causal_block=1, max_len=bound, shared=i32(common.tolist()))
    check(got, *want)


@functools.lru_cache(maxsize=1)
def shared_case(nv, seed, heads, group, dim, blocks, seqs):
    news = [n for _, n in seqs]
    pool, common = shared_pool(nv, seed, heads, dim, blocks, list(seqs))
    tables = pool.table.copy()
    tables[0, :blocks] = common
    one_dim_a_block(pool, tables)
    q = normal(gen(seed + 1), sum(news), heads * group, dim)
    rs = starts(news)
    want = step_ref.attention(q.double().numpy(), pool.ref, rs, pool.lens.tolist(), pool.table, scale_of(dim), 1, shared=common)
    return pool, common, q.cuda(), rs, want


@pytest.mark.parametrize("blocks,rows,count", [(100, 1, 9), (33, 3, 40), (300, 1, 1), (130, 40, 5)])
@pytest.mark.parametrize("dim", [64, 128])
@BOUND
def test_every_block_of_a_longer_prefix(nv, dim, blocks, rows, count, bound):
    seqs = tuple((7 * i % 150, rows) for i in range(count))
    pool, common, q, rs, want = shared_case(nv, 430, 2, 4, dim, blocks, seqs)
    check_shared(nv, pool, common, q, rs, bound, want)


@pytest.mark.parametrize("dim,heads,group,blocks,own,seqs", [
    (64, 8, 8, 128, 9600, ((1500, 8), (0, 8))),
    (64, 2, 64, 200, 9600, ((3000, 1), (10, 3), (64, 4))),
    (128, 1, 64, 400, 45000, ((2500, 10), (0, 0), (63, 6))),
])
def test_more_than_32_pieces_of_many_rows(nv, dim, heads, group, blocks, own, seqs):
    """The join in which one wave takes up to 64 parts of a row: from 1024 rows and heads on, over a prefix in many pieces and
    own keys in several."""
    pool, common, q, rs, want = shared_case(nv, 440, heads, group, dim, blocks, seqs)
    bound = blocks * BLOCK + own
    assert shared_pieces(nv, len(q), len(seqs), heads, group, dim, blocks, bound) > 32 and len(q) * heads * group >= 1024
    check_shared(nv, pool, common, q, rs, bound, want)


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("kind", ["window", "shared"])
def test_inputs_that_a_side_stream_still_makes(nv, kind, given):
    """Queries and cached keys that come late on a side stream, which the call is given or finds current; two such streams
    at once, with workspaces of their own.  A call on another stream would read what is not there yet."""
    pool, common = shared_pool(nv, 450, 2, 128, 20, [(4700, 1), (50, 1)])
    if kind == "shared":
        kw = dict(shared=i32(common.tolist()))
        assert shared_pieces(nv, 2, 2, 2, 4, 128, 20, pool.tab.shape[1] * BLOCK) > 1
    else:
        pool.tab[:, :20] = i32(common.tolist())
        kw = dict(window=4500, sinks=5)
        assert window_pieces(nv, 2, 2, 2, 4, 128, 1, 4500, 5, pool.tab.shape[1] * BLOCK) > 1
    big, rs = torch.randn(4096, 4096, device="cuda"), i32([0, 1, 2])
    sides = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        q = normal(gen(451 + turn), 2, 8, 128).cuda()
        late = [(torch.zeros_like(q), nv.KvCache(*[torch.zeros_like(t) for t in (pool.gpu.k, pool.gpu.v, pool.gpu.k_power,
                                                                                pool.gpu.v_power)])) for _ in sides]
        want = nv.kv_attention(q, pool.gpu, rs, pool.lens, pool.tab, causal_block=1, **kw)
        torch.cuda.synchronize()
        got = []
        for side, (x, cache) in zip(sides, late):
            with torch.cuda.stream(side):
                for _ in range(20):
                    y = big @ big
                x.copy_(q + 0 * y[:2, :1, None].bfloat16().nan_to_num(0))
                for a, b in ((cache.k, pool.gpu.k), (cache.v, pool.gpu.v), (cache.k_power, pool.gpu.k_power),
                             (cache.v_power, pool.gpu.v_power)):
                    torch.add(b, 0, out=a)
        for side, (x, cache) in zip(sides, late):
            with torch.cuda.stream(torch.cuda.current_stream() if given else side):
                got.append(nv.kv_attention(x, cache, rs, pool.lens, pool.tab, causal_block=1,
                                           **(dict(stream=side) if given else {}), **kw))
        assert not sides[1].query()  # the inputs were still being made
        for side, o in zip(sides, got):
            side.synchronize()
            assert same(o, want)


# ---------------------------------------------------------------------------
# the references themselves
# ---------------------------------------------------------------------------
def test_the_bound_sees_a_block_left_out(nv):
    """On the host: a reference without one of the prefix's blocks is outside the bound that the kernels are held to.  (With
    at most dim blocks each is alone in its output: left out, the output is off by itself, of which the bound is a few
    steps of 2^-8.)"""
    pool, common, q, rs, (want, tol) = shared_case(nv, 430, 2, 4, 128, 100, tuple((7 * i, 1) for i in range(9)))
    check(torch.from_numpy(want), want, tol)
    for at in (0, 37, 99):
        cache = kv_ref.Cache(pool.ref.blocks, 2, 128)
        cache.codes = [pool.ref.codes[0], pool.ref.codes[1].copy()]
        cache.powers = pool.ref.powers
        cache.codes[1][common[at]] = 0
        less, _ = step_ref.attention(q.cpu().double().numpy(), cache, rs, pool.lens.tolist(), pool.table, scale_of(128), 1,
                                     shared=common)
        with pytest.raises(AssertionError, match="outside"):
            check(torch.from_numpy(less), want, tol)
