"""Python binding of the MI355X NVFP4 activation producer and block-scaled GEMM.

Argument marshalling only: every step of the path runs in the HIP kernels of
``libnvfp4.so`` (built in-tree by ``build.py``).  PyTorch provides device
memory and the current stream.  There is no fallback: importing this package
without the built library raises.

Functions named like the C entry points (``nvfp4_modulate_absmax`` ...) take
torch tensors and the same arguments as the C ABI (``include/nvfp4.h``);
``modulate_quantize``, ``swiglu_quantize`` and ``gemm`` are conveniences that
allocate their outputs with torch, and so are ``rope_table``, ``rope``,
``KvCache``, ``kv_write``, ``kv_read`` and ``kv_attention`` for what lies between
the QKV projection and the attention output's quantizer, with ``norm_rope`` for
the norms of its heads and ``KvStep``, ``kv_extend`` and ``kv_release`` for the
tables that the cache's calls take.
"""
from __future__ import annotations

import ctypes
import os

import torch  # loads the HIP runtime that the library must share

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

NVFP4_OK = 0
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "misaligned pointer or stride",
           4: "invalid segment table", 5: "HIP launch failure"}
MAX_SEGMENTS = 16


class Nvfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int, hip_error: int = 0):
        msg = f"{fn}: {_STATUS.get(status, status)}"
        if status == 5:
            msg += f" (hip error {hip_error})"
        super().__init__(msg)
        self.status = status


class Segments(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("row_start", ctypes.POINTER(ctypes.c_int64)),
                ("shift", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class RowGates(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("row_start", ctypes.POINTER(ctypes.c_int64)),
                ("gate", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


ROPE_MAX_AXES = 4
KV_BLOCK = 64


class RopeParams(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("split", ctypes.c_int32), ("pairs", ctypes.c_int32 * ROPE_MAX_AXES),
                ("rows", ctypes.c_int64 * ROPE_MAX_AXES), ("table", ctypes.c_void_p * ROPE_MAX_AXES),
                ("positions", ctypes.c_void_p), ("ld_positions", ctypes.c_int64)]


class KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_power", ctypes.c_void_p),
                ("v_power", ctypes.c_void_p), ("blocks", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32)]


class KvSequences(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("row_start", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("table_blocks", ctypes.c_int64)]


class KvTables(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("table_blocks", ctypes.c_int64), ("free_blocks", ctypes.c_void_p), ("capacity", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run nvfp4_activation_quantization_segment_amd/build.py")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, V = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    SEG = ctypes.POINTER(Segments)
    GATES = ctypes.POINTER(RowGates)
    HEADS, ROPE = ctypes.POINTER(Heads), ctypes.POINTER(RopeParams)
    CACHE, SEQS, TABLES = ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvSequences), ctypes.POINTER(KvTables)
    sigs = {
        "nvfp4_padded_rows": (I64, [I64]),
        "nvfp4_absmax_workspace_bytes": (ctypes.c_size_t, []),
        "nvfp4_set_barrier_timeout_us": (ctypes.c_uint64, [ctypes.c_uint64]),
        "nvfp4_set_barrier_help_us": (ctypes.c_uint64, [ctypes.c_uint64]),
        "nvfp4_modulate_absmax": (I32, [P, I64, I64, I64, SEG, P, P, P, V]),
        "nvfp4_modulate_pack": (I32, [P, I64, I64, I64, SEG, P, P, P, I64, V]),
        "nvfp4_modulate_quantize": (I32, [P, I64, I64, I64, SEG, P, P, P, P, P, I64, V]),
        "nvfp4_modulate_quantize_noalloc": (I32, [P, I64, I64, I64, SEG, P, P, P, P, I64, V]),
        "nvfp4_quantize": (I32, [P, I64, I64, I64, P, P, P, P, P, I64, V]),
        "nvfp4_swiglu_absmax": (I32, [P, P, I64, I64, I64, P, P, P, V]),
        "nvfp4_swiglu_pack": (I32, [P, P, I64, I64, I64, P, P, P, I64, V]),
        "nvfp4_swiglu_quantize": (I32, [P, P, I64, I64, I64, P, P, P, P, P, I64, V]),
        "nvfp4_gemm": (I32, [P, P, P, I64, I64, P, P, P, I64, I64, P, I64, V]),
        "nvfp4_gemm_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64]),
        "nvfp4_gemm_ws": (I32, [P, P, P, I64, I64, P, P, P, I64, I64, P, I64, P, ctypes.c_size_t, V]),
        "nvfp4_gemm_gate_residual": (I32, [P, P, P, I64, I64, P, P, P, I64, I64, GATES, P, I64, P, I64, P,
                                            ctypes.c_size_t, V]),
        "nvfp4_ring_slot_bytes": (ctypes.c_size_t, [I64, I64]),
        "nvfp4_ring_gemm_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I64]),
        "nvfp4_modulate_gemm_ring": (I32, [P, I64, I64, I64, SEG, P, P, P, P, I32, I64, P, P, P, I64, P, I64, P,
                                           ctypes.c_size_t, V]),
        "nvfp4_rope_table": (I32, [P, I64, I32, ctypes.c_double, V]),
        "nvfp4_rope": (I32, [HEADS, I64, I32, I32, ROPE, HEADS, V]),
        "nvfp4_kv_write": (I32, [CACHE, SEQS, I64, HEADS, HEADS, ROPE, V]),
        "nvfp4_kv_read": (I32, [CACHE, SEQS, I64, HEADS, HEADS, V]),
        "nvfp4_kv_attention_workspace_bytes": (ctypes.c_size_t, [I64, I64, I32, I32, I32, I64]),
        "nvfp4_kv_attention": (I32, [HEADS, I64, I32, CACHE, SEQS, ctypes.c_float, I32, I64, HEADS, P,
                                     ctypes.c_size_t, V]),
        "nvfp4_kv_attention_window_workspace_bytes": (ctypes.c_size_t, [I64, I64, I32, I32, I32, I32, I32, I32, I64]),
        "nvfp4_kv_attention_window": (I32, [HEADS, I64, I32, CACHE, SEQS, ctypes.c_float, I32, I32, I32, I64, HEADS, P,
                                            ctypes.c_size_t, V]),
        "nvfp4_kv_attention_shared_workspace_bytes": (ctypes.c_size_t, [I64, I64, I32, I32, I32, I64, I64]),
        "nvfp4_kv_attention_shared": (I32, [HEADS, I64, I32, CACHE, SEQS, P, I64, ctypes.c_float, I32, I64, HEADS, P,
                                            ctypes.c_size_t, V]),
        "nvfp4_norm_rope": (I32, [HEADS, I32, P, HEADS, I32, P, I64, I32, ctypes.c_float, ROPE, HEADS, HEADS, V]),
        "nvfp4_kv_extend_workspace_bytes": (ctypes.c_size_t, [I64]),
        "nvfp4_kv_extend": (I32, [TABLES, P, P, P, I64, P, P, P, P, P, P, P, ctypes.c_size_t, V]),
        "nvfp4_kv_release_workspace_bytes": (ctypes.c_size_t, [I64]),
        "nvfp4_kv_release": (I32, [TABLES, P, P, I64, P, P, P, P, ctypes.c_size_t, V]),
        "nvfp4_kv_release_to_prefix": (I32, [TABLES, P, P, I64, P, P, P, P, ctypes.c_size_t, V]),
        "nvfp4_kv_clear_rest": (I32, [HEADS, I64, I32, I32, P, I64, V]),
        "nvfp4_step_modulate": (I32, [P, P, P, P, I64, V]),
        "nvfp4_step_swiglu": (I32, [P, P, P, I64, V]),
        "nvfp4_step_block_scale": (I32, [P, P, P, I64, V]),
        "nvfp4_step_element_code": (I32, [P, P, P, P, I64, V]),
        "nvfp4_step_e2m1": (I32, [P, P, I64, V]),
        "nvfp4_step_e4m3": (I32, [P, P, I64, V]),
        "nvfp4_status_string": (ctypes.c_char_p, [I32]),
        "nvfp4_last_hip_error": (ctypes.c_int, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _ptr(t) -> ctypes.c_void_p | None:
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(fn: str, status: int):
    if status != NVFP4_OK:
        raise Nvfp4Error(fn, status, lib.nvfp4_last_hip_error())


def _bits16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"expected bf16 (or its 16-bit pattern), got {t.dtype}")
    return t


def make_segments(row_start, shift: torch.Tensor, scale: torch.Tensor):
    """Build the C segment table; returns (struct, keepalive)."""
    rs = (ctypes.c_int64 * len(row_start))(*[int(r) for r in row_start])
    _bits16(shift)
    _bits16(scale)
    if shift.shape != scale.shape or shift.dim() != 2 or shift.stride(1) != 1 or scale.stride(0) != shift.stride(0):
        raise ValueError("shift/scale must be [S, D] with unit column stride and equal row strides")
    seg = Segments(len(row_start) - 1, ctypes.cast(rs, ctypes.POINTER(ctypes.c_int64)), shift.data_ptr(),
                   scale.data_ptr(), shift.stride(0))
    return seg, (rs, shift, scale)


_workspaces: dict[tuple[int, int], torch.Tensor] = {}


def _torch_stream(stream, dev: torch.device):
    if stream is None:
        return torch.cuda.current_stream(dev)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=dev)


def _capturing(st) -> bool:
    """Whether work enqueued on torch stream st is being captured into a graph."""
    with torch.cuda.stream(st):
        return torch.cuda.is_current_stream_capturing()


def workspace(device=None, stream=None) -> torch.Tensor:
    """The producers' workspace for one (device, stream) pair, zero-filled on
    that stream when first made.  Calls on one stream run in order and may
    share a workspace; calls that may overlap must not (their maxima and
    barrier words would mix), so every stream gets its own."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    ts = _torch_stream(stream, dev)
    key = (dev.index, int(ts.cuda_stream))
    ws = _workspaces.get(key)
    if ws is None:
        with torch.cuda.stream(ts):
            ws = torch.zeros(int(lib.nvfp4_absmax_workspace_bytes()), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


WORKSPACE_TIMEOUT_COUNT_OFFSET = 192  # NVFP4_WORKSPACE_TIMEOUT_COUNT_OFFSET


def workspace_timeouts(ws: torch.Tensor) -> int:
    """The workspace's count of single launches whose grid-barrier wait passed
    its bound (synchronizes with the workspace's stream to read it; a caller
    that must not synchronize copies the 4 bytes asynchronously instead)."""
    o = WORKSPACE_TIMEOUT_COUNT_OFFSET
    return int(ws[o:o + 4].view(torch.int32).item())


def set_barrier_timeout_us(microseconds: int) -> int:
    """Bound on the single launches' grid-barrier wait (default 1 s); returns
    the previous bound.  0 makes every single launch give up at once."""
    return int(lib.nvfp4_set_barrier_timeout_us(int(microseconds)))


def set_barrier_help_us(microseconds: int) -> int:
    """Wait at the grid barrier before a workgroup computes absent workgroups'
    pass 1 (default 100 us); returns the previous value.  0: help at once."""
    return int(lib.nvfp4_set_barrier_help_us(int(microseconds)))


def padded_rows(m: int) -> int:
    return int(lib.nvfp4_padded_rows(int(m)))


# ---------------------------------------------------------------------------
# C entry points, same names and arguments
# ---------------------------------------------------------------------------
def nvfp4_modulate_absmax(x, M, D, ldx, seg, ws, tensor_scale, amax_out=None, stream=None):
    _check("nvfp4_modulate_absmax",
           lib.nvfp4_modulate_absmax(_ptr(x), M, D, ldx, ctypes.byref(seg), _ptr(ws), _ptr(tensor_scale),
                                     _ptr(amax_out), _stream(stream)))


def nvfp4_modulate_pack(x, M, D, ldx, seg, tensor_scale, qdata, sfa, M_pad, stream=None):
    _check("nvfp4_modulate_pack",
           lib.nvfp4_modulate_pack(_ptr(x), M, D, ldx, ctypes.byref(seg), _ptr(tensor_scale), _ptr(qdata),
                                   _ptr(sfa), M_pad, _stream(stream)))


def nvfp4_modulate_quantize(x, M, D, ldx, seg, ws, tensor_scale, amax_out, qdata, sfa, M_pad, stream=None):
    _check("nvfp4_modulate_quantize",
           lib.nvfp4_modulate_quantize(_ptr(x), M, D, ldx, ctypes.byref(seg), _ptr(ws), _ptr(tensor_scale),
                                       _ptr(amax_out), _ptr(qdata), _ptr(sfa), M_pad, _stream(stream)))


def nvfp4_modulate_quantize_noalloc(x, M, D, ldx, seg, tensor_scale, amax_out, qdata, sfa, M_pad, stream=None):
    _check("nvfp4_modulate_quantize_noalloc",
           lib.nvfp4_modulate_quantize_noalloc(_ptr(x), M, D, ldx, ctypes.byref(seg), _ptr(tensor_scale),
                                               _ptr(amax_out), _ptr(qdata), _ptr(sfa), M_pad, _stream(stream)))


def nvfp4_quantize(x, M, D, ldx, ws, tensor_scale, amax_out, qdata, sfa, M_pad, stream=None):
    _check("nvfp4_quantize",
           lib.nvfp4_quantize(_ptr(x), M, D, ldx, _ptr(ws), _ptr(tensor_scale), _ptr(amax_out), _ptr(qdata), _ptr(sfa),
                              M_pad, _stream(stream)))


def nvfp4_swiglu_absmax(gate, up, M, F, ld, ws, tensor_scale, amax_out=None, stream=None):
    _check("nvfp4_swiglu_absmax",
           lib.nvfp4_swiglu_absmax(_ptr(gate), _ptr(up), M, F, ld, _ptr(ws), _ptr(tensor_scale), _ptr(amax_out),
                                   _stream(stream)))


def nvfp4_swiglu_pack(gate, up, M, F, ld, tensor_scale, qdata, sfa, M_pad, stream=None):
    _check("nvfp4_swiglu_pack",
           lib.nvfp4_swiglu_pack(_ptr(gate), _ptr(up), M, F, ld, _ptr(tensor_scale), _ptr(qdata), _ptr(sfa), M_pad,
                                 _stream(stream)))


def nvfp4_swiglu_quantize(gate, up, M, F, ld, workspace, tensor_scale, amax, qdata, sfa, M_pad, stream=None):
    _check("nvfp4_swiglu_quantize",
           lib.nvfp4_swiglu_quantize(_ptr(gate), _ptr(up), M, F, ld, _ptr(workspace), _ptr(tensor_scale), _ptr(amax),
                                     _ptr(qdata), _ptr(sfa), M_pad, _stream(stream)))


def nvfp4_gemm(qa, sfa, a_scale, M, M_pad, qw, sfw, w_scale, N, K, out, ldo, stream=None):
    _check("nvfp4_gemm",
           lib.nvfp4_gemm(_ptr(qa), _ptr(sfa), _ptr(a_scale), M, M_pad, _ptr(qw), _ptr(sfw), _ptr(w_scale), N, K,
                          _ptr(out), ldo, _stream(stream)))


def nvfp4_gemm_workspace_bytes(M, N, K):
    return int(lib.nvfp4_gemm_workspace_bytes(M, N, K))


def nvfp4_gemm_ws(qa, sfa, a_scale, M, M_pad, qw, sfw, w_scale, N, K, out, ldo, workspace, workspace_bytes,
                  stream=None):
    _check("nvfp4_gemm_ws",
           lib.nvfp4_gemm_ws(_ptr(qa), _ptr(sfa), _ptr(a_scale), M, M_pad, _ptr(qw), _ptr(sfw), _ptr(w_scale), N, K,
                             _ptr(out), ldo, _ptr(workspace), workspace_bytes, _stream(stream)))


def make_row_gates(row_start, gate: torch.Tensor):
    """Build the C gate table; returns (struct, keepalive)."""
    rs = (ctypes.c_int64 * len(row_start))(*[int(r) for r in row_start])
    _bits16(gate)
    if gate.dim() != 2 or gate.stride(1) != 1:
        raise ValueError("gate must be [S, N] with unit column stride")
    g = RowGates(len(row_start) - 1, ctypes.cast(rs, ctypes.POINTER(ctypes.c_int64)), gate.data_ptr(), gate.stride(0))
    return g, (rs, gate)


def nvfp4_gemm_gate_residual(qa, sfa, a_scale, M, M_pad, qw, sfw, w_scale, N, K, gates, residual, ldr, out, ldo,
                             workspace, workspace_bytes, stream=None):
    _check("nvfp4_gemm_gate_residual",
           lib.nvfp4_gemm_gate_residual(_ptr(qa), _ptr(sfa), _ptr(a_scale), M, M_pad, _ptr(qw), _ptr(sfw),
                                        _ptr(w_scale), N, K, ctypes.byref(gates), _ptr(residual), ldr, _ptr(out), ldo,
                                        _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_ring_slot_bytes(chunk_rows, K):
    return int(lib.nvfp4_ring_slot_bytes(chunk_rows, K))


def nvfp4_ring_gemm_workspace_bytes(M, chunk_rows, N, K):
    return int(lib.nvfp4_ring_gemm_workspace_bytes(M, chunk_rows, N, K))


def nvfp4_modulate_gemm_ring(x, M, K, ldx, seg, ws, tensor_scale, amax_out, ring, slots, chunk_rows, qw, sfw,
                             w_scale, N, out, ldo, gemm_workspace, gemm_workspace_bytes, stream=None):
    _check("nvfp4_modulate_gemm_ring",
           lib.nvfp4_modulate_gemm_ring(_ptr(x), M, K, ldx, ctypes.byref(seg), _ptr(ws), _ptr(tensor_scale),
                                        _ptr(amax_out), _ptr(ring), slots, chunk_rows, _ptr(qw), _ptr(sfw),
                                        _ptr(w_scale), N, _ptr(out), ldo, _ptr(gemm_workspace),
                                        gemm_workspace_bytes, _stream(stream)))


# The rotary, cache and attention entry points take the structures Heads,
# RopeParams, KvCacheStruct, KvSequences and KvTables (make_heads,
# make_rope_params, KvCache.struct, make_kv_sequences, make_kv_tables); their
# tensors must outlive the call.
def nvfp4_rope_table(table, rows, pairs, theta, stream=None):
    _check("nvfp4_rope_table", lib.nvfp4_rope_table(_ptr(table), rows, pairs, theta, _stream(stream)))


def nvfp4_rope(x, M, heads, dim, rope, out, stream=None):
    _check("nvfp4_rope", lib.nvfp4_rope(x, M, heads, dim, rope, out, _stream(stream)))


def nvfp4_kv_write(cache, seqs, M, k, v, rope=None, stream=None):
    _check("nvfp4_kv_write", lib.nvfp4_kv_write(cache, seqs, M, k, v, rope, _stream(stream)))


def nvfp4_kv_read(cache, seqs, M, k, v, stream=None):
    _check("nvfp4_kv_read", lib.nvfp4_kv_read(cache, seqs, M, k, v, _stream(stream)))


def nvfp4_kv_attention_workspace_bytes(M, count, q_heads, heads, dim, max_len):
    return int(lib.nvfp4_kv_attention_workspace_bytes(M, count, q_heads, heads, dim, max_len))


def nvfp4_kv_attention(q, M, q_heads, cache, seqs, scale, causal_block, max_len, out, workspace, workspace_bytes,
                       stream=None):
    _check("nvfp4_kv_attention",
           lib.nvfp4_kv_attention(q, M, q_heads, cache, seqs, scale, causal_block, max_len, out, _ptr(workspace),
                                  workspace_bytes, _stream(stream)))


def nvfp4_kv_attention_window_workspace_bytes(M, count, q_heads, heads, dim, causal_block, window, sinks, max_len):
    return int(lib.nvfp4_kv_attention_window_workspace_bytes(M, count, q_heads, heads, dim, causal_block, window, sinks,
                                                             max_len))


def nvfp4_kv_attention_window(q, M, q_heads, cache, seqs, scale, causal_block, window, sinks, max_len, out, workspace,
                              workspace_bytes, stream=None):
    _check("nvfp4_kv_attention_window",
           lib.nvfp4_kv_attention_window(q, M, q_heads, cache, seqs, scale, causal_block, window, sinks, max_len, out,
                                         _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_kv_attention_shared_workspace_bytes(M, count, q_heads, heads, dim, shared_blocks, max_len):
    return int(lib.nvfp4_kv_attention_shared_workspace_bytes(M, count, q_heads, heads, dim, shared_blocks, max_len))


def nvfp4_kv_attention_shared(q, M, q_heads, cache, seqs, shared, shared_blocks, scale, causal_block, max_len, out,
                              workspace, workspace_bytes, stream=None):
    _check("nvfp4_kv_attention_shared",
           lib.nvfp4_kv_attention_shared(q, M, q_heads, cache, seqs, _ptr(shared), shared_blocks, scale, causal_block,
                                         max_len, out, _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_norm_rope(q, q_heads, q_weight, k, k_heads, k_weight, M, dim, eps, rope, q_out, k_out, stream=None):
    _check("nvfp4_norm_rope",
           lib.nvfp4_norm_rope(q, q_heads, _ptr(q_weight), k, k_heads, _ptr(k_weight), M, dim, eps, rope, q_out, k_out,
                               _stream(stream)))


def nvfp4_kv_extend_workspace_bytes(count):
    return int(lib.nvfp4_kv_extend_workspace_bytes(count))


def nvfp4_kv_extend(tables, past, more, free_count, M, row_start, lens, free_left, missing, positions, slots, workspace,
                    workspace_bytes, stream=None):
    _check("nvfp4_kv_extend",
           lib.nvfp4_kv_extend(tables, _ptr(past), _ptr(more), _ptr(free_count), M, _ptr(row_start), _ptr(lens),
                               _ptr(free_left), _ptr(missing), _ptr(positions), _ptr(slots), _ptr(workspace),
                               workspace_bytes, _stream(stream)))


def nvfp4_kv_release_workspace_bytes(count):
    return int(lib.nvfp4_kv_release_workspace_bytes(count))


def nvfp4_kv_release(tables, lens, done, keep, free_count, lens_out, free_left, workspace, workspace_bytes, stream=None):
    _check("nvfp4_kv_release",
           lib.nvfp4_kv_release(tables, _ptr(lens), _ptr(done), keep, _ptr(free_count), _ptr(lens_out), _ptr(free_left),
                                _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_kv_release_to_prefix(tables, lens, done, keep, free_count, lens_out, free_left, workspace, workspace_bytes,
                               stream=None):
    _check("nvfp4_kv_release_to_prefix",
           lib.nvfp4_kv_release_to_prefix(tables, _ptr(lens), _ptr(done), keep, _ptr(free_count), _ptr(lens_out),
                                          _ptr(free_left), _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_kv_clear_rest(out, M, heads, dim, row_start, count, stream=None):
    _check("nvfp4_kv_clear_rest", lib.nvfp4_kv_clear_rest(out, M, heads, dim, _ptr(row_start), count, _stream(stream)))


def nvfp4_step_modulate(x, scale, shift, y, n, stream=None):
    _check("nvfp4_step_modulate",
           lib.nvfp4_step_modulate(_ptr(x), _ptr(scale), _ptr(shift), _ptr(y), n, _stream(stream)))


def nvfp4_step_swiglu(g, u, h, n, stream=None):
    _check("nvfp4_step_swiglu", lib.nvfp4_step_swiglu(_ptr(g), _ptr(u), _ptr(h), n, _stream(stream)))


def nvfp4_step_block_scale(a16, s_g, sf, n, stream=None):
    _check("nvfp4_step_block_scale", lib.nvfp4_step_block_scale(_ptr(a16), _ptr(s_g), _ptr(sf), n, _stream(stream)))


def nvfp4_step_element_code(y, sf, s_g, code, n, stream=None):
    _check("nvfp4_step_element_code",
           lib.nvfp4_step_element_code(_ptr(y), _ptr(sf), _ptr(s_g), _ptr(code), n, _stream(stream)))


def nvfp4_step_e2m1(v, code, n, stream=None):
    _check("nvfp4_step_e2m1", lib.nvfp4_step_e2m1(_ptr(v), _ptr(code), n, _stream(stream)))


def nvfp4_step_e4m3(t, code, n, stream=None):
    _check("nvfp4_step_e4m3", lib.nvfp4_step_e4m3(_ptr(t), _ptr(code), n, _stream(stream)))


# ---------------------------------------------------------------------------
# conveniences (torch allocates the outputs)
# ---------------------------------------------------------------------------
def modulate_quantize(x: torch.Tensor, row_start, shift: torch.Tensor, scale: torch.Tensor, m_pad: int | None = None,
                      stream=None, single_pass: bool = True):
    """x [M, D] bf16 -> (qdata [M_pad, D/2] u8, sfa [M_pad, D/16] u8, tensor_scale f32[1], amax f32[1]).

    single_pass: one nvfp4_modulate_quantize launch; else nvfp4_modulate_absmax
    then nvfp4_modulate_pack (identical bytes).  Under graph capture the two
    launches are used either way: the single launch's barrier tag comes from
    the host when it is enqueued, so a replay would meet the previous replay's
    words, while the two-pass words return to zero after every call."""
    _bits16(x)
    M, D = x.shape
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    m_pad = padded_rows(M) if m_pad is None else m_pad
    seg, keep = make_segments(row_start, shift, scale)
    dev = x.device
    st = _torch_stream(stream, dev)
    with torch.cuda.stream(st):  # outputs belong to the stream that writes them
        ts = torch.empty(1, dtype=torch.float32, device=dev)
        amax = torch.empty(1, dtype=torch.float32, device=dev)
        q = torch.empty((m_pad, D // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((m_pad, D // 16), dtype=torch.uint8, device=dev)
    if single_pass and not _capturing(st):
        nvfp4_modulate_quantize(x, M, D, x.stride(0), seg, workspace(dev, st), ts, amax, q, s, m_pad, st)
    else:
        nvfp4_modulate_absmax(x, M, D, x.stride(0), seg, workspace(dev, st), ts, amax, st)
        nvfp4_modulate_pack(x, M, D, x.stride(0), seg, ts, q, s, m_pad, st)
    del keep
    return q, s, ts, amax


def swiglu_quantize(gu: torch.Tensor, m_pad: int | None = None, stream=None, combined: bool = True):
    """gate/up [M, 2F] bf16 (gate = first F columns) -> (qdata, sfa, tensor_scale, amax).

    combined: one nvfp4_swiglu_quantize call; else nvfp4_swiglu_absmax then
    nvfp4_swiglu_pack (identical bytes); the latter under graph capture, as in
    modulate_quantize."""
    _bits16(gu)
    M, F2 = gu.shape
    F = F2 // 2
    if gu.stride(1) != 1:
        raise ValueError("gate/up must have unit column stride")
    m_pad = padded_rows(M) if m_pad is None else m_pad
    dev = gu.device
    st = _torch_stream(stream, dev)
    with torch.cuda.stream(st):
        ts = torch.empty(1, dtype=torch.float32, device=dev)
        amax = torch.empty(1, dtype=torch.float32, device=dev)
        q = torch.empty((m_pad, F // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((m_pad, F // 16), dtype=torch.uint8, device=dev)
    up = gu.data_ptr() + F * gu.element_size()
    if combined and not _capturing(st):
        nvfp4_swiglu_quantize(gu, up, M, F, gu.stride(0), workspace(dev, st), ts, amax, q, s, m_pad, st)
    else:
        nvfp4_swiglu_absmax(gu, up, M, F, gu.stride(0), workspace(dev, st), ts, amax, st)
        nvfp4_swiglu_pack(gu, up, M, F, gu.stride(0), ts, q, s, m_pad, st)
    return q, s, ts, amax


_identity: dict[tuple[int, int], tuple[torch.Tensor, torch.Tensor]] = {}


def _identity_modulation(dev: torch.device, D: int, st):
    """shift = -0 and scale = +0 rows of width D (y = bf16(bf16(x * 1) + -0) = x
    for every bf16 x), kept for the life of the process: a graph that captured
    a call reads them on every replay."""
    key = (dev.index, D)
    if key not in _identity:
        with torch.cuda.stream(st):
            _identity[key] = (torch.full((1, D), -0.0, dtype=torch.bfloat16, device=dev),
                              torch.zeros((1, D), dtype=torch.bfloat16, device=dev))
    return _identity[key]


def quantize(x: torch.Tensor, m_pad: int | None = None, stream=None):
    """Plain quantizer: x [M, D] bf16 -> (qdata [M_pad, D/2], sfa [M_pad, D/16], tensor_scale f32[1], amax f32[1]).

    Under graph capture (see modulate_quantize) it runs the two modulation
    passes with the identity modulation, scale +0 and shift -0, which leaves
    every bf16 value as it is: the same bytes."""
    _bits16(x)
    M, D = x.shape
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    m_pad = padded_rows(M) if m_pad is None else m_pad
    dev = x.device
    st = _torch_stream(stream, dev)
    with torch.cuda.stream(st):
        ts = torch.empty(1, dtype=torch.float32, device=dev)
        amax = torch.empty(1, dtype=torch.float32, device=dev)
        q = torch.empty((m_pad, D // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((m_pad, D // 16), dtype=torch.uint8, device=dev)
    if _capturing(st):
        shift0, scale0 = _identity_modulation(dev, D, st)
        seg, keep = make_segments([0, M], shift0, scale0)
        nvfp4_modulate_absmax(x, M, D, x.stride(0), seg, workspace(dev, st), ts, amax, st)
        nvfp4_modulate_pack(x, M, D, x.stride(0), seg, ts, q, s, m_pad, st)
        del keep
    else:
        nvfp4_quantize(x, M, D, x.stride(0), workspace(dev, st), ts, amax, q, s, m_pad, st)
    return q, s, ts, amax


def quantize_weight(w: torch.Tensor, stream=None):
    """Prepack a bf16 weight [N, K] to NVFP4 with the plain quantizer: returns
    (qw [N, K/2], sfw [N, K/16], w_scale f32[1])."""
    N, K = w.shape
    q, s, ts, _ = quantize(w, stream=stream)
    return q[:N], s[:N], ts


def gemm(qa, sfa, a_scale, M: int, qw, sfw, w_scale, out: torch.Tensor | None = None, stream=None,
         workspace: torch.Tensor | None = None):
    """out [M, N] bf16 = bf16(a_scale * w_scale * dequant(qa) dequant(qw)^T).

    Runs nvfp4_gemm_ws on `stream` (default: the current stream); a workspace
    of nvfp4_gemm_workspace_bytes(M, N, K) bytes is allocated with torch when
    none is given.  The output and that workspace are allocated on the stream
    the GEMM runs on, so the caching allocator hands the workspace to no other
    stream's allocation before the GEMM has finished with it."""
    M_pad, Kh = qa.shape
    N = qw.shape[0]
    K = 2 * Kh
    st = _torch_stream(stream, qa.device)
    need = nvfp4_gemm_workspace_bytes(M, N, K)
    with torch.cuda.stream(st):
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=qa.device)
    nvfp4_gemm_ws(qa, sfa, a_scale, M, M_pad, qw, sfw, w_scale, N, K, out, out.stride(0), workspace,
                  need, st)
    return out


def modulate_gemm_ring(x: torch.Tensor, row_start, shift: torch.Tensor, scale: torch.Tensor, qw, sfw, w_scale,
                       chunk_rows: int = 2048, slots: int = 2, out: torch.Tensor | None = None, stream=None,
                       ring: torch.Tensor | None = None):
    """Producer + GEMM through the packed-tile ring: x [M, K] bf16 -> out [M, N]
    bf16; returns (out, tensor_scale f32[1], amax f32[1], ring).  The ring
    (slots x nvfp4_ring_slot_bytes(chunk_rows, K) bytes) and the GEMM
    workspace are allocated on the launch stream unless a ring is given."""
    _bits16(x)
    M, K = x.shape
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    N = qw.shape[0]
    seg, keep = make_segments(row_start, shift, scale)
    dev = x.device
    st = _torch_stream(stream, dev)
    slot = nvfp4_ring_slot_bytes(chunk_rows, K)
    need = nvfp4_ring_gemm_workspace_bytes(M, chunk_rows, N, K)
    with torch.cuda.stream(st):
        ts = torch.empty(1, dtype=torch.float32, device=dev)
        amax = torch.empty(1, dtype=torch.float32, device=dev)
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if ring is None or ring.numel() * ring.element_size() < slots * slot:
            ring = torch.empty(slots * slot, dtype=torch.uint8, device=dev)
        gws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    nvfp4_modulate_gemm_ring(x, M, K, x.stride(0), seg, workspace(dev, st), ts, amax, ring, slots, chunk_rows, qw,
                             sfw, w_scale, N, out, out.stride(0), gws, need, st)
    del keep
    return out, ts, amax, ring


# ---------------------------------------------------------------------------
# rotary positions, the 8-bit key/value cache and attention over it
# ---------------------------------------------------------------------------
# These checks run before every launch of a few microseconds, so they look at
# each property once and build their messages only when something is wrong.
def _same_device(dev: torch.device, *tensors):
    if dev.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {dev}")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"a tensor is on {t.device}, expected {dev}")


def make_heads(name: str, x: torch.Tensor, shape=None) -> Heads:
    """The C description of heads [rows, heads, dim] (bf16, unit stride along dim); `name` is for its messages."""
    got = x.shape
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected bf16, got {x.dtype}")
    if len(got) != 3 or (shape is not None and got != shape):
        raise ValueError(f"{name}: expected {'[rows, heads, dim]' if shape is None else list(shape)}, got {list(got)}")
    row, head, unit = x.stride()
    if unit != 1 and got[2] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    # the stride of a dimension of one element says nothing
    return Heads(x.data_ptr(), row if got[0] > 1 else 0, head if got[1] > 1 else 0)


def make_rope_params(tables, positions: torch.Tensor, rows: int, split: bool, dev: torch.device) -> RopeParams:
    """The C description of rotary positions: one [positions, pairs, 2] table for each axis, positions [rows, axes]."""
    axes = len(tables)
    if not 1 <= axes <= ROPE_MAX_AXES:
        raise ValueError(f"expected 1 to {ROPE_MAX_AXES} tables, got {axes}")
    if positions.dtype != torch.int32:
        raise TypeError(f"positions: expected int32, got {positions.dtype}")
    if positions.shape != (rows, axes) or (axes > 1 and positions.stride(1) != 1):
        raise ValueError(f"positions: expected [{rows}, {axes}] with unit stride along the last, got "
                         f"{list(positions.shape)}, strides {positions.stride()}")
    if positions.device != dev:
        raise ValueError(f"positions are on {positions.device}, expected {dev}")
    sizes, pairs, data = [], [], []
    for t in tables:
        shape = t.shape
        if t.dtype != torch.float32 or len(shape) != 3 or shape[2] != 2 or not t.is_contiguous():
            raise ValueError("a rope table is a contiguous fp32 [positions, pairs, 2]")
        if t.device != dev:
            raise ValueError(f"a rope table is on {t.device}, expected {dev}")
        sizes.append(shape[0])
        pairs.append(shape[1])
        data.append(t.data_ptr())
    return RopeParams(axes, 1 if split else 0, tuple(pairs), tuple(sizes), tuple(data), positions.data_ptr(),
                      positions.stride(0) if rows > 1 else axes)


def _empty(dev: torch.device, stream, shape, dtype=torch.bfloat16) -> torch.Tensor:
    """A new tensor of the stream that the call runs on."""
    if stream is None and dev.index == torch._C._cuda_getDevice():
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(_torch_stream(stream, dev)):
        return torch.empty(shape, dtype=dtype, device=dev)


def _output_like(name: str, t, x: torch.Tensor, stream, shape):
    """The caller's output once checked, or a new one of x's type on x's device, and its description."""
    if t is not None:
        return t, make_heads(name, t, shape)
    if stream is None:  # of the stream that is current there, which the call runs on
        t = x.new_empty(shape)
    else:
        t = _empty(x.device, stream, shape, x.dtype)
    return t, Heads(t.data_ptr(), shape[1] * shape[2], shape[2])


def _output(name: str, t, dev: torch.device, stream, shape):
    """The caller's output once checked, or a new one, and its description."""
    if t is not None:
        return t, make_heads(name, t, shape)
    t = _empty(dev, stream, shape)
    return t, Heads(t.data_ptr(), shape[1] * shape[2], shape[2])


def _call(name: str, fn, dev: torch.device, stream, *args):
    """One call on the tensors' device: on `stream`, or on that device's current stream."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
    else:
        st = _torch_stream(stream, dev)
        if st.device != dev:
            raise ValueError(f"the stream is on {st.device}, the tensors on {dev}")
        raw = st.cuda_stream
    if dev.index != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    else:
        status = fn(*args, raw)
    if status != NVFP4_OK:
        _check(name, status)


def rope_table(positions: int, pairs: int, theta: float = 10000.0, device=None, stream=None) -> torch.Tensor:
    """(cos, sin) of p * theta^(-j / pairs) for positions p and pairs j, fp32 [positions, pairs, 2]
    (formed in binary64): the table of one axis for `rope` and `kv_write`."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    _same_device(dev)
    if not (0 < positions < 2**31 and 0 < pairs < 2**31):
        raise ValueError(f"expected positions and pairs of 1 to 2^31 - 1, got {positions} and {pairs}")
    table = _empty(dev, stream, (positions, pairs, 2), torch.float32)
    _call("nvfp4_rope_table", lib.nvfp4_rope_table, dev, stream, table.data_ptr(), positions, pairs, float(theta))
    return table


def rope(x: torch.Tensor, tables, positions: torch.Tensor, split: bool = False, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Rotates the heads x [rows, heads, dim] (bf16, any row and head strides) by their positions.

    tables: one [positions, pairs, 2] table for each axis (rope_table); positions: int32 [rows, axes].
    Pairs are neighbouring dims, or with split dims half of the rotated part apart.  out may be x."""
    dev = x.device
    _same_device(dev, out)
    hx = make_heads("x", x)
    rows, heads, dim = shape = x.shape
    r = make_rope_params(tables, positions, rows, split, dev)
    out, ho = _output("out", out, dev, stream, shape)
    if rows:
        _call("nvfp4_rope", lib.nvfp4_rope, dev, stream, hx, rows, heads, dim, r, ho)
    return out


def _norm_weight(name: str, w, dim: int, dev: torch.device):
    if w is None:
        return None
    if w.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected bf16, got {w.dtype}")
    if w.shape != (dim,) or w.stride(0) != 1:
        raise ValueError(f"{name}: expected [{dim}] with unit stride, got {list(w.shape)}")
    if w.device != dev:
        raise ValueError(f"{name} is on {w.device}, expected {dev}")
    return w.data_ptr()


def norm_rope(q: torch.Tensor, k: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
              k_weight: torch.Tensor | None = None, eps: float = 1e-6, tables=(), positions: torch.Tensor | None = None,
              split: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Root-mean-square norms of the heads q [rows, q_heads, dim] and k [rows, k_heads, dim] (bf16, any row and head
    strides), times their weights [dim] (bf16; none: ones), rotated as `rope` does where tables and positions are given.

    One launch for both; formed in binary32 and rounded once.  Returns the normed queries, with k the pair of queries
    and keys.  q_out may be q and k_out k; otherwise they overlap nothing."""
    if (positions is None) != (len(tables) == 0):
        raise ValueError("rotating the heads needs tables and positions, got " +
                         ("tables" if positions is None else "positions") + " alone")
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError("a weight or an output of the keys without keys")
    dev = q.device
    _same_device(dev, k, q_out, k_out)
    hq = make_heads("q", q)
    rows, heads, dim = shape = q.shape
    hk = ko = None
    k_heads = 0
    if k is not None:
        hk = make_heads("k", k)
        k_heads = k.shape[1]
        if k.shape[0] != rows or k.shape[2] != dim:
            raise ValueError(f"k: expected [{rows}, heads, {dim}], got {list(k.shape)}")
    wq, wk = _norm_weight("q_weight", q_weight, dim, dev), _norm_weight("k_weight", k_weight, dim, dev)
    r = None if positions is None else make_rope_params(tables, positions, rows, split, dev)
    q_out, ho = _output_like("q_out", q_out, q, stream, shape)
    if k is not None:
        k_out, ko = _output_like("k_out", k_out, k, stream, k.shape)
    if rows:
        _call("nvfp4_norm_rope", lib.nvfp4_norm_rope, dev, stream, hq, heads, wq, hk, k_heads, wk, rows, dim, float(eps), r,
              ho, ko)
    return q_out if k is None else (q_out, k_out)


class KvCache:
    """A pool of 8-bit key/value cache blocks of 64 positions, as four uint8 tensors:

    k [blocks, heads, dim / 16, 64, 16] and v [blocks, heads, 4, dim, 16], E4M3 codes in the order that the
    attention kernels read them; k_power and v_power [blocks, heads], byte b standing for 2^(b - 127).
    The tensors stay the same for the cache's life; calls take the memory that they have then."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_power: torch.Tensor, v_power: torch.Tensor):
        self._tensors = k, v, k_power, v_power
        self._describe()

    def _describe(self):
        k, v, k_power, v_power = self._tensors
        if k.dim() != 5:
            raise ValueError("k must be [blocks, heads, dim / 16, 64, 16]")
        blocks, heads, groups, block, sixteen = k.shape
        dim, u8 = 16 * groups, torch.uint8
        if not (k.dtype == v.dtype == k_power.dtype == v_power.dtype == u8):
            raise TypeError(f"expected uint8, got {[t.dtype for t in (k, v, k_power, v_power)]}")
        if (block != KV_BLOCK or sixteen != 16 or v.shape != (blocks, heads, 4, dim, 16) or
                k_power.shape != (blocks, heads) or v_power.shape != (blocks, heads) or
                not (k.is_contiguous() and v.is_contiguous() and k_power.is_contiguous() and v_power.is_contiguous())):
            raise ValueError(f"expected contiguous {[blocks, heads, groups, KV_BLOCK, 16]}, {[blocks, heads, 4, dim, 16]} "
                             f"and twice {[blocks, heads]}, got {[list(t.shape) for t in (k, v, k_power, v_power)]}")
        _same_device(k.device, v, k_power, v_power)
        self._memory = k.data_ptr(), v.data_ptr(), k_power.data_ptr(), v_power.data_ptr()
        self._struct = KvCacheStruct(*self._memory, blocks, heads, dim)

    @property
    def struct(self) -> KvCacheStruct:
        """The C description, of the memory that the tensors have now."""
        k, v, k_power, v_power = self._tensors
        if (k.data_ptr(), v.data_ptr(), k_power.data_ptr(), v_power.data_ptr()) != self._memory:
            self._describe()
        return self._struct

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_power = property(lambda self: self._tensors[2])
    v_power = property(lambda self: self._tensors[3])
    device = property(lambda self: self._tensors[0].device)
    blocks = property(lambda self: self.struct.blocks)
    heads = property(lambda self: self.struct.heads)
    dim = property(lambda self: self.struct.dim)

    @classmethod
    def empty(cls, blocks: int, heads: int, dim: int, device=None) -> "KvCache":
        """A pool of zero blocks on `device` (default: the current GPU); dim 64 or 128."""
        dev = torch.device("cuda") if device is None else torch.device(device)
        make = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=dev)  # noqa: E731
        return cls(make(blocks, heads, dim // 16, KV_BLOCK, 16), make(blocks, heads, 4, dim, 16), make(blocks, heads),
                   make(blocks, heads))


def make_kv_sequences(row_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, dev: torch.device) -> KvSequences:
    """The C description of sequences: row_start [n + 1], lens [n] and table [n, blocks], int32."""
    if not (row_start.dtype == lens.dtype == table.dtype == torch.int32):
        raise TypeError(f"row_start, lens and table: expected int32, got {row_start.dtype}, {lens.dtype} and {table.dtype}")
    if row_start.device != dev or lens.device != dev or table.device != dev:
        raise ValueError(f"row_start, lens and table are on {row_start.device}, {lens.device} and {table.device}, expected "
                         f"{dev}")
    if table.dim() != 2:
        raise ValueError(f"table: expected [sequences, blocks], got {list(table.shape)}")
    n, blocks = table.shape
    ld, unit = table.stride()
    if row_start.shape != (n + 1,) or lens.shape != (n,):
        raise ValueError(f"a table of {n} sequences needs {n + 1} row starts and {n} lengths, got {list(row_start.shape)} "
                         f"and {list(lens.shape)}")
    if (unit != 1 and blocks > 1) or row_start.stride(0) != 1 or (n > 1 and lens.stride(0) != 1):
        raise ValueError("row_start, lens and table must have unit stride along the last dimension")
    return KvSequences(n, row_start.data_ptr(), lens.data_ptr(), table.data_ptr(), ld if n > 1 else blocks, blocks)


def kv_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor, lens: torch.Tensor,
             table: torch.Tensor, tables=(), positions: torch.Tensor | None = None, split: bool = False, stream=None):
    """Quantises the new rows k and v [rows, heads, dim] (bf16) into the cache.

    Sequence b's rows are row_start[b] .. row_start[b + 1], its last positions once it holds lens[b] of them;
    table [sequences, blocks] names its cache blocks (all int32 on the GPU).  With tables and positions the keys
    are rotated on the way, as `rope` does; one without the other is refused."""
    if (positions is None) != (len(tables) == 0):
        raise ValueError("rotating the keys needs their tables and positions, got " +
                         ("tables" if positions is None else "positions") + " alone")
    dev, c = cache.device, cache.struct
    _same_device(dev, k, v)
    rows = k.shape[0]
    shape = (rows, c.heads, c.dim)
    hk, hv = make_heads("k", k, shape), make_heads("v", v, shape)
    q = make_kv_sequences(row_start, lens, table, dev)
    r = None
    if positions is not None:
        r = make_rope_params(tables, positions, rows, split, dev)
    if rows:
        _call("nvfp4_kv_write", lib.nvfp4_kv_write, dev, stream, c, q, rows, hk, hv, r)


def kv_read(cache: KvCache, rows: int, row_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
            k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """Reads the positions of `rows` rows (as kv_write addresses them) back: k and v, bf16 [rows, heads, dim]."""
    dev, c = cache.device, cache.struct
    _same_device(dev, k, v)
    q = make_kv_sequences(row_start, lens, table, dev)
    shape = (rows, c.heads, c.dim)
    k, hk = _output("k", k, dev, stream, shape)
    v, hv = _output("v", v, dev, stream, shape)
    if rows:
        _call("nvfp4_kv_read", lib.nvfp4_kv_read, dev, stream, c, q, rows, hk, hv)
    return k, v


def kv_attention(q: torch.Tensor, cache: KvCache, row_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                 scale: float | None = None, causal_block: int = 0, max_len: int | None = None,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None, window: int = 0,
                 sinks: int = 0, shared: torch.Tensor | None = None, clear_rest: bool = False) -> torch.Tensor:
    """Attention of the queries q [rows, q_heads, dim] (bf16) over their sequences' cached keys and values.

    Rows and positions as in kv_write.  causal_block: 0 for no mask, 1 for causal, c for runs of c positions that
    see one another and all before them.  scale: dim^-0.5 by default.  max_len: a bound on the lengths known to the
    host (default: what the table holds), which decides how many rows a workgroup takes and how far the keys of
    few rows are shared out over workgroups.  A workspace of nvfp4_kv_attention_workspace_bytes(...) is allocated with torch when none is given,
    on the stream that the call runs on.

    window: a row sees only its last `window` positions and the first `sinks` of the sequence (0: all; sinks need a
    window).  shared: int32 [blocks] on the GPU, the cache blocks of a prefix that all sequences begin with; they stand
    for the first entries of every table, and the rows of all sequences are taken against them together.  The new rows
    lie behind it (NaN where they do not).  Not both at once.  Their workspaces are those of
    nvfp4_kv_attention_window_workspace_bytes and nvfp4_kv_attention_shared_workspace_bytes.

    clear_rest: rows of no sequence become 0, by a launch of its own (nvfp4_kv_clear_rest).  Without it they stay as they
    were: in a new output what its memory held, in q itself norm_rope's NaN of rows at position -1.  Give it wherever
    not all rows are in use (a captured step that is made for its largest) and the output goes to `quantize`, which
    takes one scale from all rows."""
    dev, c = cache.device, cache.struct
    _same_device(dev, q, out, workspace)
    hq = make_heads("q", q)
    rows, q_heads, dim = shape = q.shape
    if dim != c.dim:
        raise ValueError(f"q has heads of {dim}, the cache of {c.dim}")
    s = make_kv_sequences(row_start, lens, table, dev)
    if max_len is None:
        max_len = table.shape[1] * KV_BLOCK
    if not 0 <= causal_block < 2**31:
        raise ValueError(f"causal_block: expected 0 to 2^31 - 1, got {causal_block}")
    if not 0 <= window < 2**31 or not 0 <= sinks < 2**31:
        raise ValueError(f"window and sinks: expected 0 to 2^31 - 1, got {window} and {sinks}")
    if sinks and not window:
        raise ValueError("first positions without a window: a row sees them anyway")
    scale = dim ** -0.5 if scale is None else float(scale)
    if shared is not None:
        if window:
            raise ValueError("a window and a shared prefix in one call")
        _int32("shared", shared, None, dev)
        name, fn, size_of = "nvfp4_kv_attention_shared", lib.nvfp4_kv_attention_shared, \
            lib.nvfp4_kv_attention_shared_workspace_bytes
        sizes, args = (shared.shape[0], max_len), (shared.data_ptr(), shared.shape[0], scale, causal_block, max_len)
    elif window:
        name, fn, size_of = "nvfp4_kv_attention_window", lib.nvfp4_kv_attention_window, \
            lib.nvfp4_kv_attention_window_workspace_bytes
        sizes, args = (causal_block, window, sinks, max_len), (scale, causal_block, window, sinks, max_len)
    else:
        name, fn, size_of = "nvfp4_kv_attention", lib.nvfp4_kv_attention, lib.nvfp4_kv_attention_workspace_bytes
        sizes, args = (max_len,), (scale, causal_block, max_len)
    out, ho = _output_like("out", out, q, stream, shape)
    if workspace is None and rows:
        need = size_of(rows, s.count, q_heads, c.heads, dim, *sizes)
        if need:
            workspace = q.new_empty((need,), dtype=torch.uint8) if stream is None else _empty(dev, stream, (need,), torch.uint8)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if rows:
        _call(name, fn, dev, stream, hq, rows, q_heads, c, s, *args, ho, None if workspace is None else workspace.data_ptr(),
              size)
        if clear_rest:
            _call("nvfp4_kv_clear_rest", lib.nvfp4_kv_clear_rest, dev, stream, ho, rows, q_heads, dim, s.row_start, s.count)
    return out


# ---------------------------------------------------------------------------
# the tables of a step, built on the GPU
# ---------------------------------------------------------------------------
def _int32(name: str, t: torch.Tensor, n: int | None, dev: torch.device) -> int:
    """Where an int32 vector on `dev` of n elements (None: any number) lies, once checked."""
    shape = t.shape
    if t.dtype != torch.int32:
        raise TypeError(f"{name}: expected int32, got {t.dtype}")
    if len(shape) != 1 or (n is not None and shape[0] != n):
        raise ValueError(f"{name}: expected {'a vector' if n is None else [n]}, got {list(shape)}")
    if t.stride(0) != 1 and shape[0] > 1:
        raise ValueError(f"{name} must have unit stride")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return t.data_ptr()


def make_kv_tables(table: torch.Tensor, free: torch.Tensor) -> KvTables:
    """The C description of block tables [requests, blocks] and a stack of free blocks [capacity], int32."""
    dev = table.device
    if table.dtype != torch.int32:
        raise TypeError(f"table: expected int32, got {table.dtype}")
    if table.dim() != 2:
        raise ValueError(f"table: expected [requests, blocks], got {list(table.shape)}")
    n, blocks = table.shape
    ld, unit = table.stride()
    if unit != 1 and blocks > 1:
        raise ValueError("table must have unit stride along its last dimension")
    return KvTables(n, table.data_ptr(), ld if n > 1 else blocks, blocks, _int32("free", free, None, dev), free.shape[0])


class KvStep:
    """What kv_extend writes, for up to `rows` rows: row_start [requests + 1], lens [requests], free_count [1] and
    missing [1], positions [rows, 1] (all int32) and slots [rows] (int64), contiguous tensors that can serve step after
    step, and a workspace of nvfp4_kv_extend_workspace_bytes(requests) bytes."""

    def __init__(self, row_start: torch.Tensor, lens: torch.Tensor, free_count: torch.Tensor, missing: torch.Tensor,
                 positions: torch.Tensor, slots: torch.Tensor, workspace: torch.Tensor):
        self._tensors = row_start, lens, free_count, missing, positions, slots, workspace
        self._describe()

    def _describe(self):
        row_start, lens, free_count, missing, positions, slots, workspace = self._tensors
        dev, n = lens.device, lens.shape[0]
        _int32("row_start", row_start, n + 1, dev)
        _int32("lens", lens, n, dev)
        _int32("free_count", free_count, 1, dev)
        _int32("missing", missing, 1, dev)
        rows = positions.shape[0]
        if positions.shape != (rows, 1) or not positions.is_contiguous():
            raise ValueError(f"positions: expected a contiguous [rows, 1], got {list(positions.shape)}")
        _int32("positions", positions[:, 0], rows, dev)
        if slots.dtype != torch.int64:
            raise TypeError(f"slots: expected int64, got {slots.dtype}")
        if slots.shape != (rows,) or not slots.is_contiguous():
            raise ValueError(f"slots: expected a contiguous [{rows}], got {list(slots.shape)}")
        _same_device(dev, slots, workspace)
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        self.device, self.requests, self.rows = dev, n, rows
        self._size = workspace.numel() * workspace.element_size()
        self._memory = tuple(t.data_ptr() for t in self._tensors)

    @property
    def memory(self) -> tuple:
        """Where the tensors lie now."""
        memory = tuple([t.data_ptr() for t in self._tensors])
        if memory != self._memory:
            self._describe()
        return memory

    row_start = property(lambda self: self._tensors[0])
    lens = property(lambda self: self._tensors[1])
    free_count = property(lambda self: self._tensors[2])
    missing = property(lambda self: self._tensors[3])
    positions = property(lambda self: self._tensors[4])
    slots = property(lambda self: self._tensors[5])
    workspace = property(lambda self: self._tensors[6])

    @classmethod
    def empty(cls, requests: int, rows: int, device=None, lens: torch.Tensor | None = None,
              free_count: torch.Tensor | None = None, stream=None) -> "KvStep":
        """New tensors for it on `device` (default: the current GPU).  For steps in place give the lengths, or the count of
        free blocks, that kv_extend also takes."""
        dev = torch.device("cuda") if device is None else torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        make = lambda *shape: _empty(dev, stream, shape, torch.int32)  # noqa: E731
        return cls(make(requests + 1), make(requests) if lens is None else lens, make(1) if free_count is None else free_count,
                   make(1), make(rows, 1), _empty(dev, stream, (rows,), torch.int64),
                   _empty(dev, stream, (nvfp4_kv_extend_workspace_bytes(requests),), torch.uint8))


def kv_extend(past: torch.Tensor, more: torch.Tensor, table: torch.Tensor, free: torch.Tensor, free_count: torch.Tensor,
              step: KvStep, stream=None) -> KvStep:
    """Gives every request its next rows, positions and cache blocks, on the GPU: returns `step`, written.

    Request b holds past[b] positions and asks for more[b].  Their rows follow one another in order, cut to the rows of
    the step; the blocks they need come from the top of the stack free[:free_count], into the table [requests, blocks]
    (in place; an entry is -1 where the stack is empty, and `missing` counts those).  step.row_start, step.lens, the
    table and step.positions are what kv_write, rope and kv_attention take; step.slots is each row's block * 64 +
    position % 64.  Rows of no request get -1 in both.  step.lens may be `past` and step.free_count `free_count`.  With
    no requests or no rows nothing is given."""
    dev = step.device
    if dev.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {dev}")
    if table.device != dev:
        raise ValueError(f"table is on {table.device}, expected {dev}")
    t, n = make_kv_tables(table, free), step.requests
    if t.count != n:
        raise ValueError(f"a table of {t.count} requests, a step of {n}")
    row_start, lens, left, missing, positions, slots, workspace = step.memory
    past_at, more_at, count_at = _int32("past", past, n, dev), _int32("more", more, n, dev), _int32("free_count", free_count, 1, dev)
    if n and step.rows:
        _call("nvfp4_kv_extend", lib.nvfp4_kv_extend, dev, stream, t, past_at, more_at, count_at, step.rows, row_start, lens,
              left, missing, positions, slots, workspace, step._size)
        return step
    # no request or no row: nothing is given
    with torch.cuda.stream(_torch_stream(stream, dev)):
        step.row_start.zero_()
        step.missing.zero_()
        if lens != past_at:
            step.lens.copy_(past)
        torch.clamp(free_count, 0, t.capacity, out=step.free_count)
        step.positions.fill_(-1)
        step.slots.fill_(-1)
    return step


def kv_release(lens: torch.Tensor, done: torch.Tensor, table: torch.Tensor, free: torch.Tensor, free_count: torch.Tensor,
               keep: int = 0, lens_out: torch.Tensor | None = None, free_count_out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None, to_prefix: bool = False):
    """Takes the blocks of finished requests (done[b] != 0) back onto the stack free[:free_count], on the GPU: returns the
    lengths, 0 for those, and the stack's size after it.

    keep: the first entries of every table that are not the request's own (a shared prefix).  to_prefix: the lengths of
    finished requests become 64 * keep instead of 0, so that the next request in their place begins behind the prefix
    that its table still names; from a length of 0 kv_extend would put new blocks over those entries, which no release
    with this `keep` gives back.  The stack grows in place;
    lens_out may be `lens` and free_count_out `free_count`.  A workspace of nvfp4_kv_release_workspace_bytes(requests)
    bytes is allocated with torch when none is given, on the stream that the call runs on."""
    dev = table.device
    if dev.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {dev}")
    t = make_kv_tables(table, free)
    n = t.count
    if not 0 <= keep < 2**31:
        raise ValueError(f"keep: expected 0 to 2^31 - 1, got {keep}")
    lens_at, done_at = _int32("lens", lens, n, dev), _int32("done", done, n, dev)
    count_at = _int32("free_count", free_count, 1, dev)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"the workspace must be contiguous and on {dev}")
    if lens_out is None:
        lens_out = lens.new_empty((n,)) if stream is None else _empty(dev, stream, (n,), torch.int32)
    if free_count_out is None:
        free_count_out = lens.new_empty((1,)) if stream is None else _empty(dev, stream, (1,), torch.int32)
    lens_out_at, left_at = _int32("lens_out", lens_out, n, dev), _int32("free_count_out", free_count_out, 1, dev)
    if not n:  # nothing to take back
        with torch.cuda.stream(_torch_stream(stream, dev)):
            torch.clamp(free_count, 0, t.capacity, out=free_count_out)
        return lens_out, free_count_out
    if workspace is None:
        need = lib.nvfp4_kv_release_workspace_bytes(n)
        if need:
            workspace = _empty(dev, stream, (need,), torch.uint8)
    name, fn = ("nvfp4_kv_release_to_prefix", lib.nvfp4_kv_release_to_prefix) if to_prefix else \
        ("nvfp4_kv_release", lib.nvfp4_kv_release)
    _call(name, fn, dev, stream, t, lens_at, done_at, keep, count_at, lens_out_at, left_at,
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.numel() * workspace.element_size())
    return lens_out, free_count_out
