"""Python binding of the C ABI in include/dllm.h (ctypes).

The functions named ``dllm_*`` marshal arguments only: torch tensors become
device pointers, the current torch stream becomes the cudaStream_t, and a
non-zero status raises ``DllmError``.  Every step of the computation runs in
the CUDA library; there is no fallback.  If the library has not been built
(``python -m block_wise_kv_gb300.build``) importing the binding still works,
but the first call raises.

The helpers below (``LayerDesc``, ``BatchLayout``, ``PagedCache``) only
allocate device memory with torch and fill the C structs.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libdllm.so")

DLLM_OK = 0
DLLM_ERR_INVALID_ARGUMENT = 1
DLLM_ERR_UNSUPPORTED = 2
DLLM_ERR_WORKSPACE_TOO_SMALL = 3
DLLM_ERR_CUDA = 4
DLLM_ERR_TIMEOUT = 5

DLLM_DEVERR_TIMEOUT = 1
DLLM_DEVERR_BAD_PAGE = 2
DLLM_DEVERR_BAD_SHAPE = 4
DLLM_DEVERR_RANGE = 8
DLLM_DEVERR_NO_PAGES = 16

DLLM_OP_CACHE_BUILD = 0
DLLM_OP_BLOCK_QKV_ROPE_WRITE = 1
DLLM_OP_BLOCK_ATTENTION = 2
DLLM_OP_STATE_MERGE = 3
DLLM_OP_STEP_ATTENTION = 4
DLLM_OP_CACHE_ADVANCE = 5

DLLM_ROWS_BLOCK = 0
DLLM_ROWS_FULL = 1

DLLM_ACT_NONE = 0
DLLM_ACT_SILU = 1
DLLM_ACT_GELU = 2
DLLM_ACT_GELU_TANH = 3

DLLM_ROPE_HALVES = 0
DLLM_ROPE_NEIGHBOURS = 1

DLLM_TYPE_BF16 = 0
DLLM_TYPE_FP32 = 1

PAGE = 64
_BF16, _FP32, _INT32 = torch.bfloat16, torch.float32, torch.int32
KV8_GROUP = 16  # token positions that share a scale of the 8-bit cache

# Every symbol include/dllm.h declares.
EXPORTS = ("dllm_workspace_size", "dllm_rope_table_build", "dllm_qkv_weight_packed_bytes", "dllm_qkv_weight_pack",
           "dllm_cache_build", "dllm_cache_advance", "dllm_block_qkv_rope_write", "dllm_block_qkv_rope_write_noalloc",
           "dllm_block_attention", "dllm_state_merge", "dllm_step_attention", "dllm_lm_head_workspace_size",
           "dllm_block_lm_head", "dllm_ffn_workspace_size", "dllm_block_ffn", "dllm_batch_plan", "dllm_kv8_write",
           "dllm_kv8_write_pool", "dllm_kv8_attention_workspace_size", "dllm_kv8_attention",
           "dllm_linear_workspace_size", "dllm_linear", "dllm_head_norm_rope", "dllm_token_scores",
           "dllm_status_string")


class DllmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({dllm_status_string(status)})")


class LayerDescC(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("softmax_scale", ctypes.c_float)]


class CacheC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("q_pool", ctypes.c_void_p),
                ("m_pool", ctypes.c_void_p), ("l_pool", ctypes.c_void_p), ("o_pool", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32),
                ("m_pre", ctypes.c_void_p), ("l_pre", ctypes.c_void_p), ("o_pre", ctypes.c_void_p)]


class BatchC(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("total_block_rows", ctypes.c_int32), ("total_seq_rows", ctypes.c_int32),
                ("max_block_len", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p), ("block_start", ctypes.c_void_p),
                ("block_len", ctypes.c_void_p), ("cu_block", ctypes.c_void_p), ("cu_seq", ctypes.c_void_p),
                ("error_flag", ctypes.c_void_p)]


class Kv8CacheC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32)]


class PageRingC(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("state", ctypes.c_void_p), ("state_out", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


class LinearLayerC(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("act", ctypes.c_int32),
                ("gated", ctypes.c_int32), ("rms_eps", ctypes.c_float)]


class HeadRowsC(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("in_row_stride", ctypes.c_int64), ("in_head_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("gain", ctypes.c_void_p), ("n_heads", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libdllm.so (raises if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"CUDA library not built: {p} is missing "
                                   "(run `python -m block_wise_kv_gb300.build`)")
            lib = ctypes.CDLL(p)
            P = ctypes.POINTER
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            sig = {
                "dllm_workspace_size": [P(LayerDescC), P(BatchC), i32, P(sz)],
                "dllm_rope_table_build": [P(LayerDescC), i32, vp, vp],
                "dllm_qkv_weight_packed_bytes": [P(LayerDescC), P(sz)],
                "dllm_qkv_weight_pack": [P(LayerDescC), vp, vp, vp],
                "dllm_cache_build": [P(LayerDescC), P(BatchC), vp, vp, vp, vp, i32, P(CacheC), vp, sz, vp],
                "dllm_cache_advance": [P(LayerDescC), P(BatchC), P(BatchC), vp, vp, vp, vp, i32, P(CacheC), vp, sz,
                                       vp],
                "dllm_block_qkv_rope_write": [P(LayerDescC), P(BatchC), vp, vp, vp, vp, i32, P(CacheC), vp, vp, sz,
                                              vp],
                "dllm_block_qkv_rope_write_noalloc": [P(LayerDescC), P(BatchC), vp, vp, vp, vp, i32, P(CacheC), vp,
                                                      vp],
                "dllm_block_attention": [P(LayerDescC), P(BatchC), vp, P(CacheC), vp, vp, vp, sz, vp],
                "dllm_state_merge": [P(LayerDescC), P(BatchC), P(CacheC), vp, vp, vp, sz, vp],
                "dllm_step_attention": [P(LayerDescC), P(BatchC), vp, P(CacheC), vp, vp, vp, sz, vp],
                "dllm_lm_head_workspace_size": [P(LayerDescC), P(BatchC), i32, P(sz)],
                "dllm_block_lm_head": [P(LayerDescC), P(BatchC), i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                "dllm_ffn_workspace_size": [P(LayerDescC), P(BatchC), i32, P(sz)],
                "dllm_block_ffn": [P(LayerDescC), P(BatchC), i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                "dllm_batch_plan": [P(BatchC), vp, vp, vp, vp, vp, P(PageRingC), vp, vp, vp, vp],
                "dllm_kv8_write": [P(LayerDescC), P(BatchC), vp, i64, i64, vp, i64, i64, P(Kv8CacheC), vp],
                "dllm_kv8_write_pool": [P(LayerDescC), P(BatchC), P(CacheC), P(Kv8CacheC), vp],
                "dllm_kv8_attention_workspace_size": [P(LayerDescC), P(BatchC), P(Kv8CacheC), P(sz)],
                "dllm_kv8_attention": [P(LayerDescC), P(BatchC), vp, i64, P(Kv8CacheC), vp, i32, vp, vp, sz, vp],
                "dllm_linear_workspace_size": [P(LinearLayerC), i32, i32, P(sz)],
                "dllm_linear": [P(LinearLayerC), i32, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, sz, vp],
                "dllm_head_norm_rope": [P(LayerDescC), i32, vp, P(HeadRowsC), P(HeadRowsC), vp, i32, i32, i32, vp, vp],
                "dllm_token_scores": [i32, i32, vp, i32, i64, ctypes.c_float, vp, vp, vp, vp, i32, vp, vp, vp, vp],
            }
            for name, argt in sig.items():
                fn = getattr(lib, name)
                fn.argtypes = argt
                fn.restype = ctypes.c_int
            lib.dllm_status_string.argtypes = [ctypes.c_int]
            lib.dllm_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the handle alone: building torch's stream object costs microseconds a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _nbytes(t) -> int:
    if t is None or isinstance(t, int):
        return 0
    return t.numel() * t.element_size()


def _check(fn: str, status: int) -> None:
    if status != DLLM_OK:
        raise DllmError(fn, status)


# ------------------------------------------------------------ the C ABI ----
def dllm_status_string(status: int) -> str:
    return load().dllm_status_string(int(status)).decode()


def dllm_workspace_size(desc: LayerDescC, batch: BatchC, op: int) -> int:
    out = ctypes.c_size_t(0)
    _check("dllm_workspace_size", load().dllm_workspace_size(ctypes.byref(desc), ctypes.byref(batch), op,
                                                             ctypes.byref(out)))
    return out.value


def dllm_rope_table_build(desc: LayerDescC, max_pos: int, rope_table: torch.Tensor, stream=None) -> None:
    _check("dllm_rope_table_build", load().dllm_rope_table_build(ctypes.byref(desc), int(max_pos), _ptr(rope_table),
                                                                 _stream(stream)))


def dllm_qkv_weight_packed_bytes(desc: LayerDescC) -> int:
    out = ctypes.c_size_t(0)
    _check("dllm_qkv_weight_packed_bytes", load().dllm_qkv_weight_packed_bytes(ctypes.byref(desc), ctypes.byref(out)))
    return out.value


def dllm_qkv_weight_pack(desc: LayerDescC, w_qkv: torch.Tensor, w_packed: torch.Tensor, stream=None) -> None:
    _check("dllm_qkv_weight_pack", load().dllm_qkv_weight_pack(ctypes.byref(desc), _ptr(w_qkv), _ptr(w_packed),
                                                               _stream(stream)))


def pack_qkv_weight(desc: LayerDescC, w_qkv: torch.Tensor, stream=None) -> torch.Tensor:
    """The tile-packed copy of a device bf16 [3*H*d][d_model] weight that the
    projection calls take (allocated here, filled by dllm_qkv_weight_pack)."""
    n = dllm_qkv_weight_packed_bytes(desc)
    out = torch.empty(n // 2, dtype=torch.bfloat16, device=w_qkv.device)
    dllm_qkv_weight_pack(desc, w_qkv.contiguous(), out, stream)
    return out


def dllm_cache_build(desc, batch, x_full, rms_gain, w_packed, rope_table, rope_max_pos, cache, ws, stream=None):
    _check("dllm_cache_build", load().dllm_cache_build(
        ctypes.byref(desc), ctypes.byref(batch), _ptr(x_full), _ptr(rms_gain), _ptr(w_packed), _ptr(rope_table),
        int(rope_max_pos), ctypes.byref(cache), _ptr(ws), _nbytes(ws), _stream(stream)))


def dllm_cache_advance(desc, batch, decoded, x_decoded, rms_gain, w_packed, rope_table, rope_max_pos, cache, ws,
                       stream=None):
    _check("dllm_cache_advance", load().dllm_cache_advance(
        ctypes.byref(desc), ctypes.byref(batch), ctypes.byref(decoded), _ptr(x_decoded), _ptr(rms_gain),
        _ptr(w_packed), _ptr(rope_table), int(rope_max_pos), ctypes.byref(cache), _ptr(ws), _nbytes(ws),
        _stream(stream)))


def dllm_block_qkv_rope_write(desc, batch, x_block, rms_gain, w_packed, rope_table, rope_max_pos, cache, q_block,
                              ws, stream=None):
    _check("dllm_block_qkv_rope_write", load().dllm_block_qkv_rope_write(
        ctypes.byref(desc), ctypes.byref(batch), _ptr(x_block), _ptr(rms_gain), _ptr(w_packed), _ptr(rope_table),
        int(rope_max_pos), ctypes.byref(cache), _ptr(q_block), _ptr(ws), _nbytes(ws), _stream(stream)))


def dllm_block_qkv_rope_write_noalloc(desc, batch, x_block, rms_gain, w_packed, rope_table, rope_max_pos, cache,
                                      q_block, stream=None):
    """dllm_block_qkv_rope_write without a workspace: for callers that cannot
    allocate device memory (the library's fixed 8 MiB scratch is used)."""
    _check("dllm_block_qkv_rope_write_noalloc", load().dllm_block_qkv_rope_write_noalloc(
        ctypes.byref(desc), ctypes.byref(batch), _ptr(x_block), _ptr(rms_gain), _ptr(w_packed), _ptr(rope_table),
        int(rope_max_pos), ctypes.byref(cache), _ptr(q_block), _stream(stream)))


def dllm_block_attention(desc, batch, q_block, cache, o_full, lse=None, ws=None, stream=None):
    _check("dllm_block_attention", load().dllm_block_attention(
        ctypes.byref(desc), ctypes.byref(batch), _ptr(q_block), ctypes.byref(cache), _ptr(o_full), _ptr(lse),
        _ptr(ws), _nbytes(ws), _stream(stream)))


def dllm_state_merge(desc, batch, cache, o_full, lse=None, ws=None, stream=None):
    _check("dllm_state_merge", load().dllm_state_merge(
        ctypes.byref(desc), ctypes.byref(batch), ctypes.byref(cache), _ptr(o_full), _ptr(lse), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def dllm_step_attention(desc, batch, q_block, cache, o_full, lse=None, ws=None, stream=None):
    _check("dllm_step_attention", load().dllm_step_attention(
        ctypes.byref(desc), ctypes.byref(batch), _ptr(q_block), ctypes.byref(cache), _ptr(o_full), _ptr(lse),
        _ptr(ws), _nbytes(ws), _stream(stream)))


def dllm_lm_head_workspace_size(desc, batch, vocab: int) -> int:
    out = ctypes.c_size_t(0)
    _check("dllm_lm_head_workspace_size", load().dllm_lm_head_workspace_size(ctypes.byref(desc), ctypes.byref(batch),
                                                                             int(vocab), ctypes.byref(out)))
    return int(out.value)


def dllm_block_lm_head(desc, batch, vocab, h_full, final_gain, w_lm, logits, lse, argmax, p_max, ws, stream=None):
    _check("dllm_block_lm_head", load().dllm_block_lm_head(
        ctypes.byref(desc), ctypes.byref(batch), int(vocab), _ptr(h_full), _ptr(final_gain), _ptr(w_lm),
        _ptr(logits), _ptr(lse), _ptr(argmax), _ptr(p_max), _ptr(ws), _nbytes(ws), _stream(stream)))


def dllm_ffn_workspace_size(desc, batch, d_ff: int) -> int:
    out = ctypes.c_size_t(0)
    _check("dllm_ffn_workspace_size", load().dllm_ffn_workspace_size(ctypes.byref(desc), ctypes.byref(batch),
                                                                     int(d_ff), ctypes.byref(out)))
    return int(out.value)


def dllm_block_ffn(desc, batch, d_ff, o_full, x_block, w_o, ffn_gain, w_gate_up, w_gate_up_scale, w_down,
                   w_down_scale, y_block, ws, stream=None):
    _check("dllm_block_ffn", load().dllm_block_ffn(
        ctypes.byref(desc), ctypes.byref(batch), int(d_ff), _ptr(o_full), _ptr(x_block), _ptr(w_o), _ptr(ffn_gain),
        _ptr(w_gate_up), _ptr(w_gate_up_scale), _ptr(w_down), _ptr(w_down_scale), _ptr(y_block), _ptr(ws),
        _nbytes(ws), _stream(stream)))


# The calls of the 8-bit cache are made for small batches too, where the host's part is most of their time: they take
# tensors only, and check type, layout, length and device once each, in as few steps as that takes.
def _on(device: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def dllm_batch_plan(batch, pages_held, pages_held_out, block_table, cu_block, cu_seq, ring, row_slot=None,
                    row_seq=None, row_pos=None, stream=None):
    """pages_held, pages_held_out: int32 [batch]; block_table [batch][max_pages_per_seq]; cu_block, cu_seq
    [batch + 1]; the row maps [total_block_rows], each may be None.  All contiguous, longer ones are fine."""
    i32, dev, n, rows = _INT32, pages_held.get_device(), 4 * batch.batch, 4 * batch.total_block_rows
    table, cub, cus = block_table.data_ptr(), cu_block.data_ptr(), cu_seq.data_ptr()
    # (written out: a helper for each tensor takes a microsecond more.  What the batch names itself is what it says.)
    if (pages_held.dtype is not i32 or pages_held.nbytes < n or not pages_held.is_contiguous()
            or pages_held_out.dtype is not i32 or pages_held_out.nbytes < n or not pages_held_out.is_contiguous()
            or pages_held_out.get_device() != dev
            or table != batch.block_table and (
                block_table.dtype is not i32 or block_table.nbytes < n * batch.max_pages_per_seq
                or not block_table.is_contiguous() or block_table.get_device() != dev)
            or cub != batch.cu_block and (cu_block.dtype is not i32 or cu_block.nbytes <= n
                                          or not cu_block.is_contiguous() or cu_block.get_device() != dev)
            or cus != batch.cu_seq and (cu_seq.dtype is not i32 or cu_seq.nbytes <= n
                                        or not cu_seq.is_contiguous() or cu_seq.get_device() != dev)
            or row_slot is not None and (row_slot.dtype is not i32 or row_slot.nbytes < rows
                                         or not row_slot.is_contiguous() or row_slot.get_device() != dev)
            or row_seq is not None and (row_seq.dtype is not i32 or row_seq.nbytes < rows
                                        or not row_seq.is_contiguous() or row_seq.get_device() != dev)
            or row_pos is not None and (row_pos.dtype is not i32 or row_pos.nbytes < rows
                                        or not row_pos.is_contiguous() or row_pos.get_device() != dev)
            or dev != torch._C._cuda_getDevice()):
        raise DllmError("dllm_batch_plan", DLLM_ERR_INVALID_ARGUMENT)
    status = (_lib or load()).dllm_batch_plan(
        batch, pages_held.data_ptr(), pages_held_out.data_ptr(), table, cub, cus, ring,
        None if row_slot is None else row_slot.data_ptr(), None if row_seq is None else row_seq.data_ptr(),
        None if row_pos is None else row_pos.data_ptr(), _on(dev, stream))
    if status:
        raise DllmError("dllm_batch_plan", status)


def dllm_kv8_write(desc, batch, k_rows: torch.Tensor, v_rows: torch.Tensor, kv8, stream=None):
    """k_rows, v_rows: bf16 [M][n_kv_heads][head_dim], M >= total_block_rows, the last dimension
    contiguous (views of a wider projection output are fine)."""
    ks, vs, shape = k_rows.stride(), v_rows.stride(), k_rows.shape
    if (len(ks) != 3 or shape != v_rows.shape or ks[2] != 1 or vs[2] != 1 or shape[1] != kv8.n_kv_heads
            or shape[2] != desc.head_dim or shape[0] < batch.total_block_rows or k_rows.dtype is not _BF16
            or v_rows.dtype is not _BF16):
        raise DllmError("dllm_kv8_write", DLLM_ERR_INVALID_ARGUMENT)
    dev = k_rows.get_device()
    if v_rows.get_device() != dev or dev != torch._C._cuda_getDevice():
        raise DllmError("dllm_kv8_write", DLLM_ERR_INVALID_ARGUMENT)
    status = (_lib or load()).dllm_kv8_write(
        desc, batch, k_rows.data_ptr(), ks[0], ks[1], v_rows.data_ptr(), vs[0], vs[1], kv8, _on(dev, stream))
    if status:
        raise DllmError("dllm_kv8_write", status)


def dllm_kv8_write_pool(desc, batch, cache, kv8, stream=None):
    status = (_lib or load()).dllm_kv8_write_pool(desc, batch, cache, kv8, _stream(stream))
    if status:
        raise DllmError("dllm_kv8_write_pool", status)


def dllm_kv8_attention_workspace_size(desc, batch, kv8) -> int:
    out = ctypes.c_size_t(0)
    _check("dllm_kv8_attention_workspace_size", load().dllm_kv8_attention_workspace_size(
        ctypes.byref(desc), ctypes.byref(batch), ctypes.byref(kv8), ctypes.byref(out)))
    return int(out.value)


def dllm_kv8_attention(desc, batch, q: torch.Tensor, kv8, o, lse, ws, o_rows: int = DLLM_ROWS_BLOCK, stream=None):
    """q: bf16 [M][n_heads][head_dim], M >= total_block_rows, rows contiguous, any row stride.  o: contiguous bf16 of
    as many rows (DLLM_ROWS_FULL: of total_seq_rows rows), lse: contiguous float32 of as many rows of n_heads, or
    None; ws: a uint8 tensor of dllm_kv8_attention_workspace_size bytes."""
    qs, shape, n_heads, d, m = q.stride(), q.shape, desc.n_heads, desc.head_dim, batch.total_block_rows
    if (len(qs) != 3 or qs[2] != 1 or shape[1] != n_heads or shape[2] != d or (qs[1] != d and n_heads > 1)
            or shape[0] < m or q.dtype is not _BF16):
        raise DllmError("dllm_kv8_attention", DLLM_ERR_INVALID_ARGUMENT)
    dev = q.get_device()
    values = (batch.total_seq_rows if o_rows == DLLM_ROWS_FULL else m) * n_heads
    if (o.dtype is not _BF16 or o.nbytes < 2 * values * d or not o.is_contiguous() or o.get_device() != dev
            or not ws.is_contiguous() or ws.get_device() != dev
            or lse is not None and (lse.dtype is not _FP32 or lse.nbytes < 4 * values or not lse.is_contiguous()
                                    or lse.get_device() != dev)
            or dev != torch._C._cuda_getDevice()):
        raise DllmError("dllm_kv8_attention", DLLM_ERR_INVALID_ARGUMENT)
    status = (_lib or load()).dllm_kv8_attention(
        desc, batch, q.data_ptr(), qs[0], kv8, o.data_ptr(), o_rows, None if lse is None else lse.data_ptr(),
        ws.data_ptr(), ws.nbytes, _on(dev, stream))
    if status:
        raise DllmError("dllm_kv8_attention", status)


def dllm_linear_workspace_size(layer, rows: int, normed: bool) -> int:
    out = ctypes.c_size_t(0)
    _check("dllm_linear_workspace_size", load().dllm_linear_workspace_size(
        ctypes.byref(layer), int(rows), int(bool(normed)), ctypes.byref(out)))
    return int(out.value)


def _vector_ok(t, dtype, n: int, dev: int) -> bool:
    """Whether t is a contiguous tensor of n values or more."""
    return t.dtype is dtype and t.numel() >= n and t.is_contiguous() and t.get_device() == dev


def dllm_linear(layer, x: torch.Tensor, w, y, rms_gain=None, bias=None, residual=None, ws=None, error=None,
                stream=None):
    """x: bf16 [M][in_features], w: contiguous bf16 [out_features (gated: twice that)][in_features], y and residual:
    bf16 [M][out_features]; x, y and residual with any row stride; rms_gain, bias: bf16 vectors; ws: a uint8 tensor of
    dllm_linear_workspace_size bytes (with a gain); error: an int32 word."""
    k, n = layer.in_features, layer.out_features
    wide = 2 * n if layer.gated else n
    shape, xs, ys, dev = x.shape, x.stride(), y.stride(), x.get_device()
    m = shape[0]
    if (shape != (m, k) or y.shape != (m, n) or w.shape != (wide, k) or x.dtype is not _BF16 or w.dtype is not _BF16
            or y.dtype is not _BF16 or xs[1] != 1 and k > 1 or ys[1] != 1 and n > 1 or not w.is_contiguous()
            or w.get_device() != dev or y.get_device() != dev
            or rms_gain is not None and not _vector_ok(rms_gain, _BF16, k, dev)
            or bias is not None and not _vector_ok(bias, _BF16, wide, dev)
            or error is not None and not _vector_ok(error, _INT32, 1, dev)
            or ws is not None and (not ws.is_contiguous() or ws.get_device() != dev)
            or dev != torch._C._cuda_getDevice()):
        raise DllmError("dllm_linear", DLLM_ERR_INVALID_ARGUMENT)
    rp, rs = None, n
    if residual is not None:
        st = residual.stride()
        if (residual.dtype is not _BF16 or residual.shape != (m, n) or st[1] != 1 and n > 1
                or residual.get_device() != dev):
            raise DllmError("dllm_linear", DLLM_ERR_INVALID_ARGUMENT)
        rp, rs = residual.data_ptr(), st[0] if m > 1 else n
    status = (_lib or load()).dllm_linear(
        layer, m, x.data_ptr(), xs[0] if m > 1 else k, None if rms_gain is None else rms_gain.data_ptr(), w.data_ptr(),
        None if bias is None else bias.data_ptr(), rp, rs, y.data_ptr(), ys[0] if m > 1 else n,
        None if error is None else error.data_ptr(), None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.nbytes, _on(dev, stream))
    if status:
        raise DllmError("dllm_linear", status)


def _head_rows(t, out, gain, m: int, d: int, dev: int):
    """The dllm_head_rows of bf16 tensors [m][heads][d], or None where they do not fit."""
    shape = t.shape
    if (len(shape) != 3 or out.shape != shape or t.dtype is not _BF16 or out.dtype is not _BF16
            or t.get_device() != dev or out.get_device() != dev):
        return None
    rows, h, width = shape
    ti, th, te = t.stride()
    oi, oh, oe = out.stride()
    if rows != m or width != d or te != 1 or oe != 1:
        return None
    if gain is None:
        g = None
    elif gain.dtype is _BF16 and gain.numel() >= d and gain.is_contiguous() and gain.get_device() == dev:
        g = gain.data_ptr()
    else:
        return None
    if m == 1:
        ti = oi = h * d
    if h == 1:
        th = oh = d
    return HeadRowsC(t.data_ptr(), ti, th, out.data_ptr(), oi, oh, g, h)


def dllm_head_norm_rope(desc, q: torch.Tensor, q_out, k, k_out, row_pos, rope_table, q_gain=None, k_gain=None,
                        pairs: int = DLLM_ROPE_HALVES, error=None, stream=None):
    """q, q_out: bf16 [M][n_heads][head_dim], k, k_out: bf16 [M][any number of heads][head_dim] or None, the last
    dimension contiguous, outputs the inputs themselves or apart from them; row_pos: contiguous int32 of M positions
    (more are fine); rope_table: contiguous float32 [positions][rotary_dim / 2][2]; gains: bf16 [head_dim] or None."""
    d, m, dev, ts = desc.head_dim, q.shape[0], torch._C._cuda_getDevice(), rope_table.shape
    queries = _head_rows(q, q_out, q_gain, m, d, dev)
    keys = None if k is None else _head_rows(k, k_out, k_gain, m, d, dev)
    if (queries is None or k is not None and keys is None or row_pos is None or row_pos.dtype is not _INT32
            or row_pos.numel() < m or not row_pos.is_contiguous() or row_pos.get_device() != dev
            or rope_table.dtype is not _FP32 or len(ts) != 3 or ts[2] != 2 or not rope_table.is_contiguous()
            or rope_table.get_device() != dev or error is not None and not _vector_ok(error, _INT32, 1, dev)):
        raise DllmError("dllm_head_norm_rope", DLLM_ERR_INVALID_ARGUMENT)
    status = (_lib or load()).dllm_head_norm_rope(
        desc, m, row_pos.data_ptr(), queries, keys, rope_table.data_ptr(), ts[0], 2 * ts[1], pairs,
        None if error is None else error.data_ptr(), _on(dev, stream))
    if status:
        raise DllmError("dllm_head_norm_rope", status)


def dllm_token_scores(logits: torch.Tensor, tokens=None, logp=None, lse=None, entropy=None, top_ids=None,
                      top_logp=None, scale: float = 1.0, error=None, stream=None):
    """logits: bf16 or float32 [M][vocab], any row stride; tokens: int32 and logp: float32 of M values, or both None;
    lse, entropy: float32 of M values or None; top_ids: contiguous int32 and top_logp: contiguous float32 [M][top_k], or
    both None."""
    dev, shape, ls, dtype = logits.get_device(), logits.shape, logits.stride(), logits.dtype
    if len(shape) != 2:
        raise DllmError("dllm_token_scores", DLLM_ERR_INVALID_ARGUMENT)
    m, vocab = shape
    top = 0 if top_ids is None else top_ids.shape[-1]
    if (dtype is not _BF16 and dtype is not _FP32 or ls[1] != 1 and vocab > 1
            or (tokens is None) != (logp is None) or (top_ids is None) != (top_logp is None)
            or top_ids is not None and (
                top_ids.shape != (m, top) or top_logp.shape != (m, top) or not _vector_ok(top_ids, _INT32, m * top, dev)
                or not _vector_ok(top_logp, _FP32, m * top, dev))
            or tokens is not None and (not _vector_ok(tokens, _INT32, m, dev) or not _vector_ok(logp, _FP32, m, dev))
            or lse is not None and not _vector_ok(lse, _FP32, m, dev)
            or entropy is not None and not _vector_ok(entropy, _FP32, m, dev)
            or error is not None and not _vector_ok(error, _INT32, 1, dev) or dev != torch._C._cuda_getDevice()):
        raise DllmError("dllm_token_scores", DLLM_ERR_INVALID_ARGUMENT)
    status = (_lib or load()).dllm_token_scores(
        m, vocab, logits.data_ptr(), DLLM_TYPE_BF16 if dtype is _BF16 else DLLM_TYPE_FP32, ls[0] if m > 1 else vocab,
        scale, None if tokens is None else tokens.data_ptr(), None if logp is None else logp.data_ptr(),
        None if lse is None else lse.data_ptr(), None if entropy is None else entropy.data_ptr(), top,
        None if top_ids is None else top_ids.data_ptr(), None if top_logp is None else top_logp.data_ptr(),
        None if error is None else error.data_ptr(), _on(dev, stream))
    if status:
        raise DllmError("dllm_token_scores", status)


# ---------------------------------------------------- memory / structs ----
def layer_desc(d_model: int, n_heads: int, head_dim: int, rope_theta: float, rms_eps: float = 1e-5,
               softmax_scale: float = 0.0) -> LayerDescC:
    return LayerDescC(d_model, n_heads, head_dim, PAGE, rope_theta, rms_eps, softmax_scale)


def linear_desc(in_features: int, out_features: int, act: int = DLLM_ACT_NONE, gated: bool = False,
                rms_eps: float = 1e-5) -> LinearLayerC:
    return LinearLayerC(in_features, out_features, act, int(gated), rms_eps)


class BatchLayout:
    """Device copies of the batch metadata and the dllm_batch struct that
    points at them (the tensors stay alive as long as this object)."""

    def __init__(self, block_table, seq_len, block_start, block_len, device="cuda", error_flag: bool = True):
        bt = np.asarray(block_table, dtype=np.int32)
        self.host = dict(block_table=bt, seq_len=np.asarray(seq_len, np.int32),
                         block_start=np.asarray(block_start, np.int32), block_len=np.asarray(block_len, np.int32))
        h = self.host
        h["cu_block"] = np.concatenate([[0], np.cumsum(h["block_len"])]).astype(np.int32)
        h["cu_seq"] = np.concatenate([[0], np.cumsum(h["seq_len"])]).astype(np.int32)
        self.batch = int(h["seq_len"].shape[0])
        self.dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(device) for k, v in h.items()}
        self.error = torch.zeros(1, dtype=torch.int32, device=device) if error_flag else None
        self.max_pages = int(bt.shape[1]) if bt.ndim == 2 and bt.shape[1] > 0 else 1
        self.total_block_rows = int(h["cu_block"][-1])
        self.total_seq_rows = int(h["cu_seq"][-1])
        self.max_block_len = int(h["block_len"].max()) if self.batch else 1
        self.max_seq_len = int(h["seq_len"].max()) if self.batch else 1
        d = self.dev
        self.c = BatchC(self.batch, self.max_pages, self.total_block_rows, self.total_seq_rows, self.max_block_len,
                        self.max_seq_len, _ptr(d["block_table"]), _ptr(d["seq_len"]), _ptr(d["block_start"]),
                        _ptr(d["block_len"]), _ptr(d["cu_block"]), _ptr(d["cu_seq"]), _ptr(self.error))

    def error_bits(self) -> int:
        return 0 if self.error is None else int(self.error.item())

    def with_blocks(self, block_start, block_len) -> "BlockRange":
        """The same sequences with other block ranges (for dllm_cache_advance's
        decoded blocks): the struct shares this layout's block table, seq_len,
        cu_seq and error flag."""
        return BlockRange(self, block_start, block_len)


class BlockRange:
    """A dllm_batch that shares a BatchLayout's sequences and points at its own
    block_start / block_len / cu_block."""

    def __init__(self, base: BatchLayout, block_start, block_len):
        bs = np.asarray(block_start, np.int32)
        bl = np.asarray(block_len, np.int32)
        cu = np.concatenate([[0], np.cumsum(bl)]).astype(np.int32)
        dev = base.dev["seq_len"].device
        self.host = dict(block_start=bs, block_len=bl, cu_block=cu)
        self.dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(dev) for k, v in self.host.items()}
        self.total_block_rows = int(cu[-1])
        self.max_block_len = int(bl.max()) if bl.size else 1
        d, bd = self.dev, base.dev
        self.c = BatchC(base.batch, base.max_pages, self.total_block_rows, base.total_seq_rows, self.max_block_len,
                        base.max_seq_len, _ptr(bd["block_table"]), _ptr(bd["seq_len"]), _ptr(d["block_start"]),
                        _ptr(d["block_len"]), _ptr(d["cu_block"]), _ptr(bd["cu_seq"]), _ptr(base.error))


class BatchView:
    """A dllm_batch over device tensors that the caller holds (int32, as
    dllm_batch_plan fills them), with the host bounds that size the launches.
    The tensors stay alive as long as this object."""

    def __init__(self, block_table, seq_len, block_start, block_len, cu_block, cu_seq, total_block_rows: int,
                 total_seq_rows: int, max_block_len: int, max_seq_len: int, error=None):
        self.tensors = (block_table, seq_len, block_start, block_len, cu_block, cu_seq, error)
        self.error = error
        for t in self.tensors:
            if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
                raise ValueError("batch metadata are contiguous int32 tensors")
            if t is not None and t.device != seq_len.device:
                raise ValueError("batch metadata are tensors of one device")
        n = seq_len.numel()
        if (seq_len.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] < n or block_start.numel() < n
                or block_len.numel() < n or cu_block.numel() <= n or cu_seq.numel() <= n
                or error is not None and error.numel() < 1):
            raise ValueError("batch metadata are seq_len, block_start, block_len [batch], block_table [batch][pages], "
                             "cu_block and cu_seq [batch + 1], and one error word")
        self.c = BatchC(seq_len.shape[0], block_table.shape[1], total_block_rows, total_seq_rows, max_block_len,
                        max_seq_len, _ptr(block_table), _ptr(seq_len), _ptr(block_start), _ptr(block_len),
                        _ptr(cu_block), _ptr(cu_seq), _ptr(error))

    def error_bits(self) -> int:
        return 0 if self.error is None else int(self.error.item())


class PageRing:
    """A dllm_page_ring over device int32 tensors: pages [P], state [2] (head,
    count) and state_out [2]."""

    def __init__(self, pages, state, state_out):
        for t in (pages, state, state_out):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("a page ring's tensors are contiguous int32")
            if t.device != pages.device:
                raise ValueError("a page ring's tensors are of one device")
        if pages.dim() != 1 or state.numel() < 2 or state_out.numel() < 2:
            raise ValueError("a page ring has pages [P], state [2] and state_out [2]")
        self.pages, self.state, self.state_out = pages, state, state_out
        self.c = PageRingC(_ptr(pages), _ptr(state), _ptr(state_out), pages.shape[0])

    @classmethod
    def full(cls, num_pages: int, device="cuda") -> "PageRing":
        """Every page free, in order."""
        return cls(torch.arange(num_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, num_pages], dtype=torch.int32, device=device),
                   torch.zeros(2, dtype=torch.int32, device=device))

    def swapped(self) -> "PageRing":
        """The ring of the next step: this one's state_out is its state."""
        return PageRing(self.pages, self.state_out, self.state)


class Kv8Cache:
    """The 8-bit paged pools of one layer: codes as torch.float8_e4m3fn (zero)
    and one scale per 16 positions of a head (one)."""

    def __init__(self, num_pages: int, n_kv_heads: int, head_dim: int, device="cuda", tensors=None):
        if tensors is None:
            shape = (num_pages, n_kv_heads, PAGE, head_dim)
            k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
            ks, vs = (torch.ones(num_pages, n_kv_heads, PAGE // KV8_GROUP, device=device) for _ in range(2))
            tensors = (k, v, ks, vs)
        self.k, self.v, self.k_scale, self.v_scale = tensors
        for t, dtype in zip(tensors, (torch.float8_e4m3fn,) * 2 + (torch.float32,) * 2):
            if t.dtype != dtype or not t.is_contiguous():
                raise ValueError("the pools are contiguous float8_e4m3fn tensors, the scales contiguous float32")
            if t.device != self.k.device:
                raise ValueError("the pools and their scales are of one device")
        shape = (num_pages, n_kv_heads, PAGE, head_dim)
        scales = (num_pages, n_kv_heads, PAGE // KV8_GROUP)
        if any(tuple(t.shape) != s for t, s in zip(tensors, (shape, shape, scales, scales))):
            raise ValueError(f"pools of shape {shape} and scales of shape {scales} are needed")
        self.num_pages = num_pages
        self.c = Kv8CacheC(_ptr(self.k), _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale), num_pages, n_kv_heads)

    @classmethod
    def of(cls, k, v, k_scale, v_scale) -> "Kv8Cache":
        """Over tensors that the caller holds."""
        return cls(k.shape[0], k.shape[1], k.shape[3], tensors=(k, v, k_scale, v_scale))


class PagedCache:
    """The paged pools of one layer, allocated by torch (zero-filled, or
    filled with `fill` to act as a sentinel)."""

    def __init__(self, num_pages: int, n_heads: int, head_dim: int, device="cuda", fill: float | None = None,
                 pre: bool = False):
        shp = (num_pages, n_heads, PAGE, head_dim)

        def mk(shape, dtype):
            t = torch.zeros(shape, dtype=dtype, device=device)
            if fill is not None:
                t.fill_(fill)
            return t

        self.k = mk(shp, torch.bfloat16)
        self.v = mk(shp, torch.bfloat16)
        self.q = mk(shp, torch.bfloat16)
        self.m = mk(shp[:3], torch.float32)
        self.l = mk(shp[:3], torch.float32)
        self.o = mk(shp, torch.float16)  # the state's O~ / l
        self.num_pages = num_pages
        # the prefix state (for incremental boundaries), when asked for
        self.m_pre = mk(shp[:3], torch.float32) if pre else None
        self.l_pre = mk(shp[:3], torch.float32) if pre else None
        self.o_pre = mk(shp, torch.float16) if pre else None
        self.c = CacheC(_ptr(self.k), _ptr(self.v), _ptr(self.q), _ptr(self.m), _ptr(self.l), _ptr(self.o),
                        num_pages, _ptr(self.m_pre), _ptr(self.l_pre), _ptr(self.o_pre))


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Caller-owned scratch of at least nbytes (256-byte aligned by torch's
    allocator), zero-filled."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def gather_rows(pool: torch.Tensor, block_table: np.ndarray, b: int, n: int) -> torch.Tensor:
    """Rows 0..n-1 of sequence b from a pool [P, H, 64, ...] -> [n, H, ...]
    (a torch index operation, for tests and inspection)."""
    pos = torch.arange(n)
    pages = torch.from_numpy(np.asarray(block_table[b], dtype=np.int64))[pos // PAGE].to(pool.device)
    slots = (pos % PAGE).to(pool.device)
    return pool[pages, :, slots]
