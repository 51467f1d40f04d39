"""CPU tests of the operators around the cache: refusals (nothing is launched), the workspaces, the binding's checks and
structures, and the index arithmetic of windows, compiled from the header that the kernels use."""
import ctypes
import os
import subprocess

import pytest
import torch

from tests import kv_ref, step_ref
from tests.test_attention_abi import (ALIGNMENT, CACHE_ERRORS, CSRC, FAKE, HEADS_ERRORS, INVALID, OVERLAPS, ROOT, ROPE_ERRORS,
                                      ROWS_ERRORS, SEQ_ERRORS, SHAPE, cache, heads, rope, seqs)


@pytest.fixture(scope="module")
def nv():
    import nvfp4_activation_quantization_segment_amd as m

    return m


def tables(nv, count=2, table=FAKE, ld=4, blocks=4, free=FAKE, capacity=8):
    return nv.KvTables(count, table, ld, blocks, free, capacity)


TABLE_ERRORS = [(dict(table=None), INVALID), (dict(free=None), INVALID), (dict(count=0), INVALID), (dict(blocks=0), INVALID),
                (dict(ld=3), INVALID), (dict(capacity=0), INVALID), (dict(count=(1 << 20) + 1), SHAPE),
                (dict(ld=1 << 26, blocks=1 << 26), SHAPE), (dict(ld=1 << 60), SHAPE), (dict(capacity=(1 << 30) + 1), SHAPE),
                (dict(table=FAKE + 2), ALIGNMENT), (dict(free=FAKE + 1), ALIGNMENT)]


def test_norm_rope_refusals(nv):
    f = nv.lib.nvfp4_norm_rope

    def call(q=None, qh=8, qw=FAKE, k="yes", kh=4, kw=FAKE, M=10, d=128, eps=1e-6, r="yes", qo=None, ko="yes"):
        return f(q or heads(nv), qh, qw, heads(nv) if k == "yes" else k, kh, kw, M, d, eps, rope(nv) if r == "yes" else r,
                 qo or heads(nv), heads(nv) if ko == "yes" else ko, None)

    for bad, want in HEADS_ERRORS:
        for name in ("q", "k", "qo", "ko"):
            assert call(**{name: heads(nv, **bad)}) == want, (name, bad)
    for bad in OVERLAPS:
        assert call(qo=heads(nv, **bad)) == INVALID, bad
    assert call(ko=heads(nv, row=384)) == INVALID and call(ko=heads(nv, head=120)) == INVALID
    for bad, want in ROPE_ERRORS:
        assert call(r=rope(nv, **bad)) == want, bad
    for M, want in ROWS_ERRORS:
        assert call(M=M) == want, M
    for eps in (0.0, -1e-6, 1e-39, 1.0001, float("inf"), float("nan")):
        assert call(eps=eps) == INVALID, eps
    assert call(qh=0) == INVALID and call(kh=-1) == INVALID and call(qh=65536) == SHAPE and call(kh=65536) == SHAPE
    assert call(d=0) == INVALID and call(d=120) == SHAPE and call(d=528) == SHAPE
    assert call(qw=FAKE + 8) == ALIGNMENT and call(kw=FAKE + 2) == ALIGNMENT
    # no keys: nothing of theirs
    assert call(k=None) == INVALID and call(ko=None) == INVALID
    for bad in (dict(k=None, ko=None), dict(k=None, kw=None), dict(ko=None, kw=None)):
        assert call(kh=0, **bad) == INVALID, bad
    assert call(q=heads(nv, data=None), kh=0, k=None, ko=None, kw=None) == INVALID


def test_extend_refusals(nv):
    f = nv.lib.nvfp4_kv_extend
    names = ("past", "more", "free_count", "M", "row_start", "lens", "free_left", "missing", "positions", "slots", "ws", "size")
    good = dict(zip(names, [FAKE, FAKE, FAKE, 10, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20]))
    call = lambda t=None, **kw: f(t or tables(nv), *[{**good, **kw}[n] for n in names], None)  # noqa: E731
    for bad, want in TABLE_ERRORS:
        assert call(tables(nv, **bad)) == want, bad
    for name in ("past", "more", "free_count", "row_start", "lens", "free_left", "missing"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: FAKE + 2}) == ALIGNMENT, name
    assert call(positions=FAKE + 2) == ALIGNMENT and call(slots=FAKE + 4) == ALIGNMENT
    for M, want in ROWS_ERRORS:
        assert call(M=M) == want, M
    need = nv.nvfp4_kv_extend_workspace_bytes(2)
    assert need > 0 and call(ws=None) == INVALID and call(size=need - 1) == INVALID and call(ws=FAKE + 8) == ALIGNMENT
    assert f(None, *[good[n] for n in names], None) == INVALID
    for count in (0, -1, (1 << 20) + 1):
        assert nv.nvfp4_kv_extend_workspace_bytes(count) == 0 and nv.nvfp4_kv_release_workspace_bytes(count) == 0


def test_release_refusals(nv):
    f = nv.lib.nvfp4_kv_release
    names = ("lens", "done", "keep", "free_count", "lens_out", "free_left", "ws", "size")
    good = dict(zip(names, [FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 1 << 20]))
    call = lambda t=None, **kw: f(t or tables(nv), *[{**good, **kw}[n] for n in names], None)  # noqa: E731
    for bad, want in TABLE_ERRORS:
        assert call(tables(nv, **bad)) == want, bad
    for name in ("lens", "done", "free_count", "lens_out", "free_left"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: FAKE + 1}) == ALIGNMENT, name
    assert call(keep=-1) == INVALID
    # a few requests need none
    assert nv.nvfp4_kv_release_workspace_bytes(1) == 0
    need, many = nv.nvfp4_kv_release_workspace_bytes(1000), tables(nv, count=1000)
    assert need > 0 and call(many, ws=None) == INVALID and call(many, size=need - 1) == INVALID
    assert call(many, ws=FAKE + 8) == ALIGNMENT
    assert f(None, *[good[n] for n in names], None) == INVALID


def test_release_to_prefix_refuses_what_release_does(nv):
    f = nv.lib.nvfp4_kv_release_to_prefix
    names = ("lens", "done", "keep", "free_count", "lens_out", "free_left", "ws", "size")
    good = dict(zip(names, [FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 1 << 20]))
    call = lambda t=None, **kw: f(t or tables(nv), *[{**good, **kw}[n] for n in names], None)  # noqa: E731
    for bad, want in TABLE_ERRORS:
        assert call(tables(nv, **bad)) == want, bad
    for name in ("lens", "done", "free_count", "lens_out", "free_left"):
        assert call(**{name: None}) == INVALID and call(**{name: FAKE + 2}) == ALIGNMENT, name
    assert call(keep=-1) == INVALID and f(None, *[good[n] for n in names], None) == INVALID
    need, many = nv.nvfp4_kv_release_workspace_bytes(1000), tables(nv, count=1000)
    assert call(many, ws=None) == INVALID and call(many, size=need - 1) == INVALID and call(many, ws=FAKE + 8) == ALIGNMENT


def test_clear_rest_refusals(nv):
    f = nv.lib.nvfp4_kv_clear_rest
    call = lambda out=None, M=10, h=8, d=128, rs=FAKE, n=2: f(out or heads(nv), M, h, d, rs, n, None)  # noqa: E731
    for bad, want in HEADS_ERRORS:
        assert call(heads(nv, **bad)) == want, bad
    for bad in OVERLAPS:
        assert call(heads(nv, **bad)) == INVALID, bad
    for M, want in ROWS_ERRORS:
        assert call(M=M) == want, M
    assert call(h=0) == INVALID and call(M=1 << 23, h=33) == SHAPE and call(M=1, h=(1 << 28) + 1) == SHAPE
    assert call(d=0) == INVALID and call(d=120) == SHAPE and call(d=528) == SHAPE
    assert call(rs=None) == INVALID and call(rs=FAKE + 2) == ALIGNMENT
    assert call(n=0) == INVALID and call(n=(1 << 20) + 1) == SHAPE
    assert f(None, 10, 8, 128, FAKE, 2, None) == INVALID


@pytest.mark.parametrize("kind", ["window", "shared"])
def test_attention_refusals(nv, kind):
    def call(q=None, M=10, q_heads=8, c=None, s=None, scale=0.1, causal=1, max_len=64, out=None, ws=FAKE, size=1 << 40,
             window=9, sinks=2, shared=FAKE, blocks=3):
        args = (q or heads(nv), M, q_heads, c or cache(nv), s or seqs(nv))
        rest = (max_len, out or heads(nv), ws, size, None)
        if kind == "window":
            return nv.lib.nvfp4_kv_attention_window(*args, scale, causal, window, sinks, *rest)
        return nv.lib.nvfp4_kv_attention_shared(*args, shared, blocks, scale, causal, *rest)

    for bad, want in HEADS_ERRORS:
        assert call(q=heads(nv, **bad)) == want and call(out=heads(nv, **bad)) == want, bad
    for bad in OVERLAPS:
        assert call(out=heads(nv, **bad)) == INVALID, bad
    for bad, want in CACHE_ERRORS:
        assert call(c=cache(nv, **bad)) == want, bad
    for bad, want in SEQ_ERRORS:
        assert call(s=seqs(nv, **bad)) == want, bad
    for M, want in ROWS_ERRORS:
        assert call(M=M) == want, M
    assert call(q_heads=0) == INVALID and call(q_heads=9) == SHAPE and call(M=1 << 23, q_heads=64) == SHAPE
    assert call(causal=-1) == INVALID and call(max_len=-1) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=scale) == INVALID, scale
    if kind == "window":
        assert call(window=0) == INVALID and call(window=-1) == INVALID and call(sinks=-1) == INVALID
        f = nv.nvfp4_kv_attention_window_workspace_bytes
        sizes = lambda **kw: f(*[{**dict(M=1, count=1, q=32, h=8, d=128, c=1, w=8000, s=4, n=1 << 20), **kw}[x]  # noqa: E731
                                 for x in ("M", "count", "q", "h", "d", "c", "w", "s", "n")])
        need = sizes()
        assert need > 0 and sizes(w=0) == sizes(s=-1) == sizes(c=-1) == sizes(M=0) == sizes(d=96) == sizes(q=33) == 0
        # more of the past than a window reaches changes nothing; without a causal mask it does
        assert sizes(n=1 << 40) == need and sizes(c=0, n=1 << 15) > sizes(c=0, n=100) == 0
        big = dict(M=1, q_heads=32, c=cache(nv, heads=8), s=seqs(nv, count=1), max_len=1 << 20, window=8000, sinks=4,
                   q=heads(nv, row=4096), out=heads(nv, row=4096))
        assert call(**big, ws=None) == INVALID and call(**big, size=need - 1) == INVALID
        assert call(**big, ws=FAKE + 8) == ALIGNMENT
    else:
        assert call(shared=None) == INVALID and call(blocks=0) == INVALID and call(blocks=-1) == INVALID
        assert call(blocks=1 << 25) == SHAPE and call(shared=FAKE + 2) == ALIGNMENT
        need = nv.nvfp4_kv_attention_shared_workspace_bytes(10, 2, 8, 8, 128, 3, 64)
        assert need >= 2 * 10 * 8 * 130 * 4
        assert call(ws=None) == INVALID and call(size=need - 1) == INVALID and call(ws=FAKE + 8) == ALIGNMENT
        f = nv.nvfp4_kv_attention_shared_workspace_bytes
        assert f(10, 2, 8, 8, 128, 0, 64) == f(10, 2, 8, 8, 128, 1 << 25, 64) == f(0, 2, 8, 8, 128, 3, 64) == 0


def test_any_prefix_has_a_plan(nv):
    """At most 48 pieces, of the prefix and of the sequences' own keys, for every size."""
    f = nv.nvfp4_kv_attention_shared_workspace_bytes
    for M in (1, 7, 33, 64, 1000, 1 << 20):
        for count in (1, 50, 5000, 1 << 20):
            for q, h, d in ((1, 1, 64), (32, 8, 128), (56, 56, 128), (255, 255, 64)):
                for blocks in (1, 2, 3, 63, 1000, (1 << 25) - 1):
                    for max_len in (0, 64 * blocks + 1, 1 << 31, (1 << 63) - 1):
                        if M * q > 1 << 28:
                            continue
                        parts, rest = divmod(f(M, count, q, h, d, blocks, max_len), M * q * (d + 2) * 4)
                        assert rest == 0 and 2 <= parts <= 48, (M, count, q, h, d, blocks, max_len)


def test_python_checks(nv):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="on a GPU"):
        nv.norm_rope(bf(2, 2, 64))
    with pytest.raises(ValueError, match="tables alone"):
        nv.norm_rope(bf(2, 2, 64), tables=[torch.zeros(4, 8, 2)])
    with pytest.raises(ValueError, match="positions alone"):
        nv.norm_rope(bf(2, 2, 64), positions=i32(2, 1))
    with pytest.raises(ValueError, match="without keys"):
        nv.norm_rope(bf(2, 2, 64), k_weight=bf(64))
    dev = torch.device("cpu")
    with pytest.raises(TypeError, match="q_weight: expected bf16"):
        nv._norm_weight("q_weight", torch.zeros(64), 64, dev)
    with pytest.raises(ValueError, match=r"q_weight: expected \[64\]"):
        nv._norm_weight("q_weight", bf(32), 64, dev)
    with pytest.raises(ValueError, match="unit stride"):
        nv._norm_weight("q_weight", bf(128)[::2], 64, dev)
    for t, error, match in ((i32(3).long(), TypeError, "int32"), (i32(4), ValueError, r"expected \[3\]"),
                            (i32(3, 1), ValueError, r"expected \[3\]"), (i32(6)[::2], ValueError, "unit stride")):
        with pytest.raises(error, match=match):
            nv._int32("lens", t, 3, dev)
    assert nv._int32("one", i32(2)[::2], 1, dev)
    with pytest.raises(TypeError, match="table: expected int32"):
        nv.make_kv_tables(i32(2, 3).long(), i32(4))
    with pytest.raises(ValueError, match="table: expected"):
        nv.make_kv_tables(i32(6), i32(4))
    with pytest.raises(ValueError, match="unit stride"):
        nv.make_kv_tables(i32(2, 6)[:, ::2], i32(4))
    with pytest.raises(TypeError, match="free: expected int32"):
        nv.make_kv_tables(i32(2, 3), i32(4).long())
    t = nv.make_kv_tables(i32(2, 6)[:, :4], i32(5))
    assert (t.count, t.ld_table, t.table_blocks, t.capacity) == (2, 6, 4, 5)
    with pytest.raises(ValueError, match="on a GPU"):
        nv.kv_release(i32(2), i32(2), i32(2, 3), i32(4), i32(1))


def test_a_step_describes_what_it_has(nv, monkeypatch):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    monkeypatch.setattr(nv, "_same_device", lambda dev, *t: None)
    make = lambda **kw: nv.KvStep(*{**dict(row_start=i32(4), lens=i32(3), free_count=i32(1), missing=i32(1),  # noqa: E731
                                           positions=i32(7, 1), slots=torch.zeros(7, dtype=torch.int64),
                                           workspace=torch.zeros(64, dtype=torch.uint8)), **kw}.values())
    s = make()
    assert (s.requests, s.rows) == (3, 7) and s.memory[1] == s.lens.data_ptr()
    for bad, error in ((dict(row_start=i32(3)), ValueError), (dict(free_count=i32(2)), ValueError),
                       (dict(missing=torch.zeros(1)), TypeError), (dict(positions=i32(7)), (ValueError, IndexError)),
                       (dict(positions=i32(7, 2)), ValueError), (dict(positions=i32(14, 1)[::2]), ValueError),
                       (dict(slots=i32(7)), TypeError), (dict(slots=torch.zeros(6, dtype=torch.int64)), ValueError),
                       (dict(workspace=torch.zeros(64, dtype=torch.uint8)[::2]), ValueError)):
        with pytest.raises(error):
            make(**bad)
    with pytest.raises(AttributeError):
        s.lens = i32(3)
    # memory that a tensor has taken since is seen
    s.lens.set_(i32(3))
    assert s.memory[1] == s.lens.data_ptr()
    s.lens.set_(i32(5))
    with pytest.raises(ValueError):
        s.memory


def test_structs_match_the_header(nv, tmp_path):
    t = nv.KvTables
    body = 'printf("%zu", sizeof(nvfp4_kv_tables));' + "".join(f'printf(" %zu", offsetof(nvfp4_kv_tables, {f[0]}));'
                                                              for f in t._fields_)
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text(f'#include <stdio.h>\n#include "{ROOT}/include/nvfp4.h"\nint main(void) {{ {body} return 0; }}\n')
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(exe)], check=True)
    size, *at = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert ctypes.sizeof(t) == int(size) and [getattr(t, f[0]).offset for f in t._fields_] == [int(a) for a in at]


def test_blocks_of_a_window(tmp_path):
    """Every block with a key that some row of a tile sees is among those it goes over, in order, and no block without
    one (of the rows' own windows, first positions and limits), over many tiles."""
    src = tmp_path / "w.cc"
    src.write_text(f'''
#include <cstdio>
#include "{CSRC}/kv_layout.h"
using namespace nvfp4;
int main() {{
    long long n, low, sinks, pos, window;
    while (scanf("%lld %lld %lld %lld %lld", &n, &low, &sinks, &pos, &window) == 5) {{
        const KvWindowBlocks b = kv_window_blocks((int)n, (int)low, (int)sinks);
        printf("%d %d %d %d\\n", b.count, b.first, b.skipped, kv_window_low((int)pos, (int)window));
    }}
}}
''')
    exe = tmp_path / "w"
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", str(src), "-o", str(exe)], check=True)
    cases, wants = [], []
    for length in (1, 63, 64, 65, 200, 700):
        for rows in (1, 5, 130):
            if rows > length:
                continue
            for causal in (1, 0, 100):
                for window in (1, 2, 63, 64, 65, 150, 1000, 2**31 - 1):
                    for sinks in (0, 1, 64, 65, 130, 2**31 - 1):
                        first = length - rows
                        low = max(0, first + 1 - window)
                        seen = max(kv_ref.limit(p, length, causal) for p in (first, length - 1))
                        n = -(-seen // 64)
                        cases.append((n, low, sinks, first, window))
                        keys = set()
                        for p in {first, length - 1, first + rows // 2}:
                            keys |= set(step_ref.visible(p, length, causal, window, sinks).nonzero()[0].tolist())
                        wants.append((low, n, sinks, sorted({k // 64 for k in keys})))
    got = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                         check=True).stdout.strip().split("\n")
    assert len(got) == len(cases)
    for line, (low, n, sinks, blocks) in zip(got, wants):
        count, first, skipped, at = map(int, line.split())
        assert at == low
        mine = [i if i < first else i + skipped for i in range(count)]
        assert set(blocks) <= set(mine) and mine == sorted(set(mine)) and (not mine or mine[-1] == n - 1)
        assert all(b * 64 < sinks or (b + 1) * 64 > low for b in mine)
