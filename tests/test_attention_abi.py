"""CPU tests of the rotary, cache and attention entry points: refusals (nothing is launched), the workspace rule, and
the index arithmetic of the cache layout and the work units, compiled from the header that the kernels use."""
import ctypes
import os
import subprocess

import pytest

from tests import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_activation_quantization_segment_amd", "csrc")
FAKE = 1 << 20  # never dereferenced: every call below fails validation first
OK, INVALID, SHAPE, ALIGNMENT = 0, 1, 2, 3


@pytest.fixture(scope="module")
def nv():
    import nvfp4_activation_quantization_segment_amd as m

    return m


def heads(nv, data=FAKE, row=1024, head=128):
    return nv.Heads(data, row, head)


def rope(nv, axes=2, pairs=(8, 8), rows=(4, 4), table=FAKE, positions=FAKE, ld=None):
    p = nv.RopeParams()
    p.axes = axes
    for a in range(min(axes, 4)) if axes > 0 else ():
        p.pairs[a], p.rows[a], p.table[a] = pairs[a % len(pairs)], rows[a % len(rows)], table
    p.positions, p.ld_positions = positions, axes if ld is None else ld
    return p


def cache(nv, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, blocks=4, heads=8, dim=128):
    return nv.KvCacheStruct(k, v, kp, vp, blocks, heads, dim)


def seqs(nv, count=2, row_start=FAKE, lens=FAKE, table=FAKE, ld=4, blocks=4):
    return nv.KvSequences(count, row_start, lens, table, ld, blocks)


HEADS_ERRORS = [(dict(data=None), INVALID), (dict(row=-8), INVALID), (dict(head=-8), INVALID), (dict(data=FAKE + 8), ALIGNMENT),
                (dict(row=1028), ALIGNMENT), (dict(head=132), ALIGNMENT), (dict(row=1 << 40), SHAPE)]
# as outputs: heads or rows that overlap
OVERLAPS = [dict(row=1016), dict(head=120), dict(row=0), dict(head=0), dict(row=128, head=1272)]
ROPE_ERRORS = [(dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(positions=None), INVALID), (dict(ld=1), INVALID),
               (dict(table=None), INVALID), (dict(pairs=(0, 8)), SHAPE), (dict(pairs=(4, 8)), SHAPE), (dict(pairs=(64, 8)), SHAPE),
               (dict(rows=(0, 4)), SHAPE), (dict(rows=(1 << 31, 4)), SHAPE), (dict(rows=(1 << 25, 4)), SHAPE), (dict(table=FAKE + 4), ALIGNMENT),
               (dict(positions=FAKE + 2), ALIGNMENT)]
CACHE_ERRORS = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID),
                (dict(blocks=0), INVALID), (dict(heads=0), INVALID), (dict(dim=96), SHAPE), (dict(dim=256), SHAPE),
                (dict(heads=65536), SHAPE), (dict(blocks=1 << 31), SHAPE), (dict(k=FAKE + 8), ALIGNMENT), (dict(v=FAKE + 4), ALIGNMENT)]
SEQ_ERRORS = [(dict(count=0), INVALID), (dict(row_start=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
              (dict(blocks=0), INVALID), (dict(ld=3), INVALID), (dict(count=(1 << 20) + 1), SHAPE),
              (dict(ld=1 << 26, blocks=1 << 26), SHAPE), (dict(lens=FAKE + 2), ALIGNMENT), (dict(row_start=FAKE + 1), ALIGNMENT),
              (dict(table=FAKE + 2), ALIGNMENT)]
ROWS_ERRORS = [(0, INVALID), (-1, INVALID), ((1 << 23) + 1, SHAPE)]


def test_rope_refusals(nv):
    L = nv.lib
    call = lambda x=None, M=10, h=8, d=128, r=None, o=None: L.nvfp4_rope(  # noqa: E731
        x or heads(nv), M, h, d, r or rope(nv), o or heads(nv), None)
    for bad, want in HEADS_ERRORS:
        assert call(x=heads(nv, **bad)) == want, bad
        assert call(o=heads(nv, **bad)) == want, bad
    for bad in OVERLAPS:
        assert call(o=heads(nv, **bad)) == INVALID, bad
    for bad, want in ROPE_ERRORS:
        assert call(r=rope(nv, **bad)) == want, bad
    for M, want in ROWS_ERRORS:
        assert call(M=M) == want
    assert call(h=0) == INVALID and call(h=65536) == SHAPE
    assert call(d=0) == INVALID and call(d=120) == SHAPE and call(d=528) == SHAPE
    assert L.nvfp4_rope(heads(nv), 10, 8, 128, None, heads(nv), None) == INVALID


def test_rope_table_refusals(nv):
    f = nv.lib.nvfp4_rope_table
    assert f(None, 4, 4, 1e4, None) == INVALID
    assert f(FAKE, 0, 4, 1e4, None) == INVALID
    assert f(FAKE, 4, 0, 1e4, None) == INVALID
    for theta in (0.0, -1.0, float("inf"), float("nan")):
        assert f(FAKE, 4, 4, theta, None) == INVALID
    assert f(FAKE, 1 << 30, 4, 1e4, None) == SHAPE
    assert f(FAKE + 4, 4, 4, 1e4, None) == ALIGNMENT
    # rows * pairs < 2^28 exactly: 3 * 89478485 = 2^28 - 1 gets as far as the pointer
    for rows, pairs in ((89478485, 3), ((1 << 28) - 1, 1), (1, (1 << 28) - 1)):
        assert f(FAKE + 4, rows, pairs, 1e4, None) == ALIGNMENT
        assert f(FAKE + 4, rows + 1, pairs, 1e4, None) == SHAPE


def test_cache_refusals(nv):
    for f in (lambda c, s, M, k, v: nv.lib.nvfp4_kv_write(c, s, M, k, v, None, None),
              lambda c, s, M, k, v: nv.lib.nvfp4_kv_read(c, s, M, k, v, None)):
        good = dict(c=cache(nv), s=seqs(nv), M=10, k=heads(nv), v=heads(nv))
        for bad, want in CACHE_ERRORS:
            assert f(**dict(good, c=cache(nv, **bad))) == want, bad
        for bad, want in SEQ_ERRORS:
            assert f(**dict(good, s=seqs(nv, **bad))) == want, bad
        for M, want in ROWS_ERRORS:
            assert f(**dict(good, M=M)) == want, M
        for bad, want in HEADS_ERRORS:
            assert f(**dict(good, k=heads(nv, **bad))) == want, bad
            assert f(**dict(good, v=heads(nv, **bad))) == want, bad
        assert f(**dict(good, c=None)) == INVALID and f(**dict(good, s=None)) == INVALID
        assert f(**dict(good, k=None)) == INVALID and f(**dict(good, v=None)) == INVALID
    for bad in OVERLAPS:
        assert nv.lib.nvfp4_kv_read(cache(nv), seqs(nv), 10, heads(nv, **bad), heads(nv), None) == INVALID, bad
        assert nv.lib.nvfp4_kv_read(cache(nv), seqs(nv), 10, heads(nv), heads(nv, **bad), None) == INVALID, bad
    for bad, want in ROPE_ERRORS:
        assert nv.lib.nvfp4_kv_write(cache(nv), seqs(nv), 10, heads(nv), heads(nv), rope(nv, **bad), None) == want, bad


def test_attention_refusals(nv):
    def call(q=None, M=10, q_heads=8, c=None, s=None, scale=0.1, causal=1, max_len=64, out=None, ws=FAKE, size=1 << 40):
        return nv.lib.nvfp4_kv_attention(q or heads(nv), M, q_heads, c or cache(nv), s or seqs(nv), scale, causal, max_len,
                                         out or heads(nv), ws, size, None)

    for bad, want in CACHE_ERRORS:
        assert call(c=cache(nv, **bad)) == want, bad
    for bad, want in SEQ_ERRORS:
        assert call(s=seqs(nv, **bad)) == want, bad
    for M, want in ROWS_ERRORS:
        assert call(M=M) == want, M
    for bad, want in HEADS_ERRORS:
        assert call(q=heads(nv, **bad)) == want, bad
        assert call(out=heads(nv, **bad)) == want, bad
    for bad in OVERLAPS:
        assert call(out=heads(nv, **bad)) == INVALID, bad
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == INVALID
    assert call(causal=-1) == INVALID and call(max_len=-1) == INVALID
    assert call(q_heads=0) == INVALID
    assert call(q_heads=12) == SHAPE                                  # not a multiple of the cache's 8
    assert call(M=1 << 23, q_heads=40) == SHAPE                       # M * q_heads > 2^28
    need = nv.lib.nvfp4_kv_attention_workspace_bytes(1, 1, 8, 8, 128, 100000)
    one = dict(M=1, s=seqs(nv, count=1), max_len=100000)
    assert need > 0
    assert call(**one, ws=None) == INVALID
    assert call(**one, size=need - 1) == INVALID
    assert call(**one, ws=FAKE + 8, size=need) == ALIGNMENT


def test_attention_workspace(nv):
    f = nv.lib.nvfp4_kv_attention_workspace_bytes
    assert f(37810, 1, 56, 56, 128, 37810) == 0        # enough rows: the keys are not shared out
    assert f(1, 1, 8, 8, 128, 64) == 0                 # one block: nothing to share out
    for bad in ((0, 1, 8, 8, 128, 64), (1, 0, 8, 8, 128, 64), (1, 1, 9, 8, 128, 64), (1, 1, 8, 8, 96, 64),
                (1, 1, 8, 8, 128, -1), (1, 1, 8, 0, 128, 64), (1 << 24, 1, 8, 8, 128, 64)):
        assert f(*bad) == 0
    per = 8 * (128 + 2) * 4                            # one part of 8 query heads
    assert f(1, 1, 8, 8, 128, 100000) % per == 0 and f(1, 1, 8, 8, 128, 100000) >= 2 * per


def test_python_checks(nv):
    import torch

    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        nv.rope(x, [torch.zeros(4, 8, 2)], torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        nv.KvCache.empty(1, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="contiguous"):
        nv.KvCache(torch.zeros(1, 1, 4, 64, 16, dtype=torch.uint8), torch.zeros(1, 1, 4, 32, 16, dtype=torch.uint8),
                   torch.zeros(1, 1, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.uint8))


LAYOUT = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kv_layout.h"
using namespace nvfp4;
static void need(bool ok, const char* what) { if (!ok) { printf("wrong: %s\n", what); exit(1); } }
int main() {
    for (int D : {64, 128}) {
        std::vector<int> k(64 * D), v(64 * D);
        for (int t = 0; t < 64; ++t)
            for (int d = 0; d < D; ++d) {
                const int a = kv_key_offset(t, d), b = kv_value_offset(t, d, D);
                need(a >= 0 && a < 64 * D && b >= 0 && b < 64 * D, "offset");
                ++k[a], ++v[b];
                printf("%d %d %d %d %d\n", D, t, d, a, b);
            }
        for (int i = 0; i < 64 * D; ++i) need(k[i] == 1 && v[i] == 1, "every byte once");
    }
    // every sequence's units fit between its base and the next one's, for all ways to share rows out
    srand(1);
    for (int round = 0; round < 20000; ++round) {
        const int B = 1 + rand() % 6;
        const int64_t per = 1 + rand() % 9, T = (round & 1) ? 32 : 128;
        std::vector<int64_t> start(1, rand() % 3 ? 0 : rand() % 200);
        for (int b = 0; b < B; ++b) start.push_back(start.back() + (rand() % 3 ? rand() % 200 : 0));
        const int64_t M = start.back() + rand() % 3;
        for (int b = 0; b < B; ++b) {
            const RowRange r = row_range(start[b], start[b + 1], M);
            const int64_t n = r.last - r.first;
            const int64_t end = b + 1 < B ? tile_base(start[b + 1], b + 1, per, T) : tile_units(M, B, per, T);
            need((n * per + T - 1) / T <= end - tile_base(r.first, b, per, T), "tiles");
            const int64_t bend = b + 1 < B ? block_base(start[b + 1], b + 1) : block_units(M, B);
            const int64_t first = rand() % 300 - 100, len = first + n;
            const int64_t touched = n ? floor_div(len - 1, 64) - floor_div(first, 64) + 1 : 0;
            need(touched <= bend - block_base(r.first, b), "blocks");
        }
    }
    // every tile and block has one unit, found as the kernels find it (the last sequence that starts at or before
    // it), whichever way the units are counted; the other units find nothing
    for (int round = 0; round < 20000; ++round) {
        const int B = 1 + rand() % 9;
        const int64_t per = rand() % 4 ? 1 + rand() % 9 : 1 + rand() % 300, T = (round & 1) ? 32 : 128;
        const int most = rand() % 2 ? 2 : 200;
        std::vector<int64_t> start(1, rand() % 3 ? 0 : rand() % 5), pos;
        for (int b = 0; b < B; ++b) start.push_back(start.back() + (rand() % 2 ? rand() % (most + 1) : 0));
        for (int b = 0; b < B; ++b) pos.push_back(rand() % 300 - 100);
        const int64_t M = start.back() + rand() % 3 + (start.back() == 0);
        const auto check = [&](int64_t units, auto first, auto wanted, const char* what) {
            std::vector<int64_t> found(B);
            for (int64_t u = 0; u < units; ++u) {
                int b = 0;
                for (int i = 1; i < B; ++i)
                    if (first(start[i], i) <= u) b = i;
                const int64_t local = u - first(start[b], b);
                if (local >= 0 && local < wanted(b)) need(found[b]++ == local, what);
            }
            for (int b = 0; b < B; ++b) need(found[b] == wanted(b), what);
        };
        const auto rows = [&](int b) { return start[b + 1] - start[b]; };
        const auto tiles = [&](int b) { return (rows(b) * per + T - 1) / T; };
        const auto blocks = [&](int b) {
            return rows(b) ? floor_div(pos[b] + rows(b) - 1, 64) - floor_div(pos[b], 64) + 1 : 0;
        };
        const int32_t t = tiles_per_row(M, B, per, T), k = blocks_per_row(M, B);
        need(tile_first(M, B, per, T, t) <= tile_units(M, B, per, T), "fewer tiles");
        need(block_first(M, B, k) <= block_units(M, B), "fewer blocks");
        for (int32_t each : {0, (int32_t)((per + T - 1) / T)})
            check(tile_first(M, B, per, T, each), [&](int64_t r, int b) { return tile_first(r, b, per, T, each); }, tiles, "tile units");
        for (int32_t each : {0, 1})
            check(block_first(M, B, each), [&](int64_t r, int b) { return block_first(r, b, each); }, blocks, "block units");
    }
    // any row starts stay inside the rows
    const int64_t odd[] = {INT32_MIN, -5, 0, 3, 7, 100, INT32_MAX};
    for (int64_t a : odd)
        for (int64_t b : odd) {
            const RowRange r = row_range(a, b, 7);
            need(0 <= r.first && r.first <= r.last && r.last <= 7, "range");
        }
    need(kv_length_bad(-1, 4) && kv_length_bad(257, 4) && !kv_length_bad(256, 4) && !kv_length_bad(0, 4), "length");
    for (int64_t c : {0, 1, 7, 64, 1000, INT32_MAX})
        for (int64_t len = 0; len < 200; ++len)
            for (int64_t pos = -70; pos < len; ++pos) {
                int64_t want = 0;
                for (int64_t j = 0; j < len; ++j)
                    want += c == 0 || (pos >= 0 && j / c <= pos / c);
                need(kv_limit(pos, len, c) == want, "limit");
            }
    // parts cover every block once, in order
    for (int64_t n = 0; n < 70; ++n)
        for (int64_t S = 1; S < 20; ++S) {
            int64_t at = 0;
            for (int64_t s = 0; s < S; ++s) {
                const BlockRange r = kv_part(n, s, S);
                need(r.first == at || (r.first == n && r.last == n), "part");
                need(r.first <= r.last && r.last <= n, "part end");
                at = r.last;
            }
            need(at == n, "all parts");
        }
    return 0;
}
"""


def test_layout_and_units(tmp_path):
    src, exe = tmp_path / "layout.cpp", tmp_path / "layout"
    src.write_text(LAYOUT)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout[-200:] + got.stderr[-500:]
    off = {D: kv_ref.offsets(D) for D in (64, 128)}
    for line in got.stdout.split("\n")[:-1]:
        D, t, d, a, b = map(int, line.split())
        assert off[D][0][t, d] == a and off[D][1][t, d] == b


def test_reference_encoder():
    """The oracle's own encoder against torch's conversion, over every bf16 magnitude up to 448 and both signs."""
    import numpy as np
    import torch

    x = torch.arange(0, 0x43E1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for v in (x, -x):
        want = v.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(kv_ref.nearest_code(v.double().numpy()), want)


def test_structs_match_the_header(nv, tmp_path):
    """The binding's structures have the header's sizes and offsets."""
    names = {"nvfp4_heads": nv.Heads, "nvfp4_rope_params": nv.RopeParams, "nvfp4_kv_cache": nv.KvCacheStruct,
             "nvfp4_kv_sequences": nv.KvSequences}
    body = "".join(f'printf("{n} %zu", sizeof({n}));' +
                   "".join(f'printf(" %zu", offsetof({n}, {f[0]}));' for f in t._fields_) + 'printf("\\n");'
                   for n, t in names.items())
    src, exe = tmp_path / "structs.c", tmp_path / "structs"
    src.write_text(f'#include <stdio.h>\n#include "{ROOT}/include/nvfp4.h"\nint main(void) {{ {body} return 0; }}\n')
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.strip().split("\n"):
        name, size, *at = line.split()
        t = names[name]
        assert ctypes.sizeof(t) == int(size)
        assert [getattr(t, f[0]).offset for f in t._fields_] == [int(a) for a in at]


def test_any_bound_on_the_lengths(nv):
    """Lengths are below 2^31; a bound past that, up to the largest number, cuts like a long one."""
    f = nv.lib.nvfp4_kv_attention_workspace_bytes
    for M, count, q_heads in ((1, 1, 8), (40, 1, 32), (32, 32, 32)):
        want = f(M, count, q_heads, 8, 128, 1 << 31)
        assert want > 0
        for max_len in (1 << 40, (1 << 63) - 64, (1 << 63) - 1):
            assert f(M, count, q_heads, 8, 128, max_len) == want


def test_positions_without_tables_are_refused(nv):
    """Positions say that the keys are to be rotated: without tables they were written as they are."""
    import types

    import torch

    cpu = torch.device("cpu")
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    pool = types.SimpleNamespace(device=cpu, heads=1, dim=64, struct=None)
    for tables in ((), []):
        with pytest.raises(ValueError, match="tables"):
            nv.kv_write(pool, x, x, i32(0, 2), i32(2), i32([0]), tables=tables, positions=torch.zeros(2, 1, dtype=torch.int32))


def test_a_cache_describes_the_memory_that_it_has(nv, monkeypatch):
    """Calls get the pointers that the tensors have then, and nothing of a cache can be assigned."""
    import torch

    monkeypatch.setattr(nv, "_same_device", lambda dev, *tensors: None)
    shapes = (3, 2, 4, 64, 16), (3, 2, 4, 64, 16), (3, 2), (3, 2)
    make = lambda: [torch.zeros(s, dtype=torch.uint8) for s in shapes]  # noqa: E731
    tensors, other = make(), make()
    c = nv.KvCache(*tensors)
    described = lambda: [getattr(c.struct, n) for n in ("k", "v", "k_power", "v_power")]  # noqa: E731
    assert described() == [t.data_ptr() for t in tensors] and (c.struct.blocks, c.struct.heads, c.struct.dim) == (3, 2, 64)
    for name, value in zip(("k", "v", "k_power", "v_power", "blocks", "heads", "dim", "device", "struct"), other + [9, 9, 9, None, None]):
        with pytest.raises(AttributeError):
            setattr(c, name, value)
    for t, o in zip(tensors, other):  # the same tensors with other memory
        t.data = o
        assert described() == [t.data_ptr() for t in tensors]
    tensors[0].data = torch.zeros(1, 2, 4, 64, 16, dtype=torch.uint8)  # and of another size
    with pytest.raises(ValueError, match="contiguous"):
        c.struct
    four = [torch.zeros((4, *s[1:]), dtype=torch.uint8) for s in shapes]
    for t, o in zip(tensors, four):
        t.data = o
    assert described() == [t.data_ptr() for t in four] and c.struct.blocks == c.blocks == 4


def test_heads_too_far_apart_are_refused(nv):
    """Attention takes up to 2^28 query heads a call: the last one's offset has to fit 64 bits, in elements and bytes."""
    def call(M, q_heads, q, out):
        return nv.lib.nvfp4_kv_attention(q, M, q_heads, cache(nv, heads=1), seqs(nv, count=1), 0.1, 1, 64, out, FAKE, 1 << 40, None)

    misaligned = heads(nv, FAKE + 8)  # as the output: the queries have passed
    for M, q_heads, stride in ((1, 1 << 28, 1 << 38), (2, 1 << 27, 1 << 37), (2, 1 << 27, 1 << 36), (1, 1 << 28, 1 << 33)):
        far = heads(nv, head=stride)
        assert call(M, q_heads, far, misaligned) == SHAPE
        # as an output, rows 8 elements apart overlap; (2^27 - 1) 2^37 is negative in 64 bits
        assert call(M, q_heads, heads(nv), heads(nv, row=8, head=stride)) == SHAPE
    for M, q_heads, stride in ((1, 1 << 20, 1 << 38), (1, 1, 1 << 38), (1 << 23, 32, 1 << 38)):
        assert call(M, q_heads, heads(nv, head=stride), misaligned) == ALIGNMENT
    assert call(1 << 23, 32, heads(nv, row=1 << 38), misaligned) == SHAPE
    assert call(1 << 22, 32, heads(nv, row=1 << 38), misaligned) == ALIGNMENT


def test_scales_past_binary32_are_refused(nv):
    """Scores are taken in base 2: scale * log2(e) has to be finite (times a score of 0 it gave NaN)."""
    def call(scale):  # a misaligned output: a good scale gets that far
        return nv.lib.nvfp4_kv_attention(heads(nv), 10, 8, cache(nv), seqs(nv), scale, 1, 64, heads(nv, FAKE + 8), FAKE, 1 << 40, None)

    for scale in (3.4e38, 2.4e38, 2.36e38):
        assert call(scale) == INVALID
    for scale in (2.35e38, 1e30, 0.1, 1e-38, 1e-45):
        assert call(scale) == ALIGNMENT


def test_heads_of_a_workgroup(tmp_path):
    """The shapes that the head loops are tested with take as many heads as they say, the last workgroup fewer."""
    lines = []
    for heads, _, seqs, write, read in kv_ref.HEAD_LOOPS:
        M = sum(n for _, n in seqs)
        assert M > 4 * len(seqs)  # the long writer
        lines.append(f"need({heads}, block_first({M}, {len(seqs)}, blocks_per_row({M}, {len(seqs)})), {write}, {read});")
    src, exe = tmp_path / "each.cpp", tmp_path / "each"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include "kv_layout.h"\nusing namespace nvfp4;\n'
                   "static void need(int heads, int64_t units, int write, int read) {\n"
                   "    const int w = kv_heads_each(units, heads, kKvWriteHeads), r = kv_heads_each(units, heads, kKvReadHeads);\n"
                   "    if (w != write || r != read || w < 2 || r < 2 || heads % w == 0 || heads % r == 0) {\n"
                   '        printf("%d heads: %d and %d a workgroup", heads, w, r);\n        exit(1);\n    }\n}\n'
                   "int main() {\n" + "\n".join(lines) + "\n}\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout


def test_shapes_that_take_wide_tiles(tmp_path):
    """The shapes that the placement of 128-row tiles is tested with take them, with odd and even numbers of units."""
    lines = []
    for _, heads, group, _, seqs in kv_ref.WIDE_HEADS:
        assert heads % 8 == 0
        M, B = sum(n for _, n in seqs) + 2 * kv_ref.WIDE_LEAD, len(seqs)
        lines.append(f"need({M}, {B}, {group}, {heads});")
    src, exe = tmp_path / "wide.cpp", tmp_path / "wide"
    src.write_text('#include <cstdlib>\n#include <initializer_list>\n#include "kv_layout.h"\nusing namespace nvfp4;\n'
                   "static int odd = 0, even = 0;\n"
                   "static void need(int64_t M, int64_t B, int64_t group, int64_t heads) {\n"
                   "    for (int blocks : {0, (1 << 20) / kKvBlock})\n"
                   "        if (!attention_wide(M, B, group, heads, blocks)) exit(1);\n"
                   "    const int64_t units = tile_first(M, B, group, kWideRows, tiles_per_row(M, B, group, kWideRows));\n"
                   "    ++(units % 2 ? odd : even);\n}\n"
                   "int main() {\n" + "\n".join(lines) + "\nreturn odd && even ? 0 : 2;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
