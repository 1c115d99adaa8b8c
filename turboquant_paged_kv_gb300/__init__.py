"""TurboQuant paged KV cache for GB300: Python binding of libtq.

Functions carry the C ABI's names (``include/tq.h``) and only marshal
arguments: torch tensors become raw device pointers, the current CUDA stream
becomes the launch stream, and a non-OK status raises ``TQError``. Every step
of the store and the decode runs inside libtq's CUDA kernels; the first call
raises ImportError if the library is not built (there is no fallback path).
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _abi
from ._abi import (PRESET_IDS, ROPE_STYLES, TQ_DEV_BLOCK_OUT_OF_RANGE, TQ_DEV_SEQ_TOO_LONG,  # noqa: F401
                   TQ_DECODE_NOALLOC_SCRATCH_BYTES, TQ_DEV_SLOT_OUT_OF_RANGE, TQ_DEV_TIMEOUT, TQ_DEV_NOT_FINITE,
                   TQ_DTYPE_BF16, TQ_DTYPE_F16, TQ_DTYPE_F32, TQ_ERR_WORKSPACE_TOO_SMALL,
                   TQError, tq_b8_layout, tq_codebook, tq_config, tq_kv16_layout, tq_layout, tq_prod_layout,
                   TQ_PRESET_KV_BF16, TQ_PRESET_KV_F16, TQ_ROPE_HALVES, TQ_ROPE_PAIRS)



class _LazyLib:
    """libtq.so, loaded on first use (raises ImportError if it is not built)."""

    def __getattr__(self, name):
        return getattr(_abi.load(), name)


_LIB = _LazyLib()

_DTYPES = {torch.float16: TQ_DTYPE_F16, torch.bfloat16: TQ_DTYPE_BF16, torch.float32: TQ_DTYPE_F32}

__all__ = ["make_config", "tq_build_codebook", "tq_layout_for", "tq_store", "tq_decode", "tq_decode_append",
           "tq_decode_partials", "tq_decode_reduce", "tq_decode_noalloc", "tq_decode_workspace_size",
           "tq_dequant", "tq_prod_layout_for", "tq_prod_store", "tq_prod_scores_workspace_size",
           "tq_prod_scores", "tq_continue_workspace_size", "tq_continue",
           "tq_b8_layout_for", "tq_b8_store", "tq_b8_dequant", "tq_b8_decode_workspace_size", "tq_b8_decode",
           "tq_b8_continue_workspace_size", "tq_b8_continue",
           "tq_kv16_layout_for", "tq_kv16_append", "tq_kv16_decode_workspace_size", "tq_kv16_decode",
           "tq_kv16_continue_workspace_size", "tq_kv16_continue",
           "tq_status_string",
           "tq_version", "TQError", "lib_path"]


def lib_path() -> str:
    return _abi.lib_path()


TQ_FLAG_INDICES_READY = 1   # include/tq.h: seq_lens / block_table not written by the previous kernel


def make_config(preset: str | int, num_q_heads: int, num_kv_heads: int, head_dim: int = 128,
                block_size: int = 16, partition_tokens: int = 0, flags: int = 0) -> tq_config:
    pid = PRESET_IDS[preset] if isinstance(preset, str) else int(preset)
    return tq_config(pid, head_dim, block_size, num_q_heads, num_kv_heads, partition_tokens, flags)


def tq_build_codebook(head_dim: int, bits: int) -> tq_codebook:
    cb = tq_codebook()
    _abi.check("tq_build_codebook", _LIB.tq_build_codebook(head_dim, bits, ctypes.byref(cb)))
    return cb


def tq_layout_for(cfg: tq_config) -> tq_layout:
    lay = tq_layout()
    _abi.check("tq_layout_for", _LIB.tq_layout_for(ctypes.byref(cfg), ctypes.byref(lay)))
    return lay


def tq_decode_workspace_size(cfg: tq_config, batch: int, max_seq_len: int) -> int:
    return int(_LIB.tq_decode_workspace_size(ctypes.byref(cfg), batch, max_seq_len))


def tq_status_string(status: int) -> str:
    return _LIB.tq_status_string(status).decode()


def tq_version() -> int:
    return int(_LIB.tq_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _cb(cb):
    return None if cb is None else ctypes.byref(cb)


def tq_store(cfg: tq_config, cb, key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
             cache: torch.Tensor, num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
             stream=None) -> None:
    """key, value [N, n_kv, d] f16/bf16; slot_mapping [N] int64; cache uint8."""
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_store", _LIB.tq_store(
        ctypes.byref(cfg), _cb(cb), _ptr(key), _ptr(value), _DTYPES[key.dtype], key.shape[0],
        _ptr(slot_mapping), _ptr(cache), num_blocks, _ptr(dev_status), _stream(stream)))


def tq_decode(cfg: tq_config, cb, q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
              seq_lens: torch.Tensor, max_seq_len: int, out: torch.Tensor, workspace: torch.Tensor,
              scale: float = 0.0, num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
              stream=None) -> None:
    """q [B, n_q, d]; block_table [B, stride] int32; seq_lens [B] int32; out [B, n_q, d]."""
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_decode", _LIB.tq_decode(
        ctypes.byref(cfg), _cb(cb), _ptr(q), _DTYPES[q.dtype], _ptr(cache), num_blocks,
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0], max_seq_len, float(scale),
        _ptr(out), _DTYPES[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _stream(stream)))


def tq_decode_append(cfg: tq_config, cb, q: torch.Tensor, new_k: torch.Tensor, new_v: torch.Tensor,
                     cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                     out: torch.Tensor, workspace: torch.Tensor, scale: float = 0.0, num_blocks: int | None = None,
                     dev_status: torch.Tensor | None = None, stream=None) -> None:
    """One decode step with its new tokens: new_k, new_v [B, n_kv, d] (q's
    dtype) are stored at position seq_lens[b] - 1 of each sequence, then the
    decode runs over all seq_lens[b] positions (one split and one reduce
    launch, no store launch)."""
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    if new_k.dtype != q.dtype or new_v.dtype != q.dtype:
        raise ValueError("new_k and new_v must have q's dtype")
    _abi.check("tq_decode_append", _LIB.tq_decode_append(
        ctypes.byref(cfg), _cb(cb), _ptr(q), _DTYPES[q.dtype], _ptr(new_k), _ptr(new_v), _ptr(cache), num_blocks,
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0], max_seq_len, float(scale),
        _ptr(out), _DTYPES[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _stream(stream)))


def tq_decode_noalloc(cfg: tq_config, cb, q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, max_seq_len: int, out: torch.Tensor, scale: float = 0.0,
                      num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
                      stream=None) -> None:
    """tq_decode without a workspace argument: the library's fixed device array
    of TQ_DECODE_NOALLOC_SCRATCH_BYTES serves as workspace (calls whose kernels
    may overlap race on it; the first call on a device does the set-up)."""
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_decode_noalloc", _LIB.tq_decode_noalloc(
        ctypes.byref(cfg), _cb(cb), _ptr(q), _DTYPES[q.dtype], _ptr(cache), num_blocks,
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0], max_seq_len, float(scale),
        _ptr(out), _DTYPES[out.dtype], _ptr(dev_status), _stream(stream)))


def tq_decode_partials(cfg: tq_config, cb, q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, max_seq_len: int, workspace: torch.Tensor, scale: float = 0.0,
                       num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
                       stream=None) -> None:
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_decode_partials", _LIB.tq_decode_partials(
        ctypes.byref(cfg), _cb(cb), _ptr(q), _DTYPES[q.dtype], _ptr(cache), num_blocks,
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0], max_seq_len, float(scale),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream)))


def tq_decode_reduce(cfg: tq_config, seq_lens: torch.Tensor, batch: int, max_seq_len: int, bt_stride: int,
                     out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _abi.check("tq_decode_reduce", _LIB.tq_decode_reduce(
        ctypes.byref(cfg), _ptr(seq_lens), batch, max_seq_len, bt_stride, _ptr(out), _DTYPES[out.dtype],
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def tq_dequant(cfg: tq_config, cb, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               max_seq_len: int, key_out: torch.Tensor, value_out: torch.Tensor, num_blocks: int | None = None,
               dev_status: torch.Tensor | None = None, stream=None) -> None:
    """key_out, value_out [B, max_seq_len, n_kv, d] (f16, bf16 or f32), written in full."""
    if value_out.dtype != key_out.dtype:
        raise ValueError("key_out and value_out must have the same dtype")
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_dequant", _LIB.tq_dequant(
        ctypes.byref(cfg), _cb(cb), _ptr(cache), num_blocks, _ptr(block_table), block_table.shape[1],
        _ptr(seq_lens), seq_lens.shape[0], max_seq_len, _ptr(key_out), _ptr(value_out),
        _DTYPES[key_out.dtype], _ptr(dev_status), _stream(stream)))


def tq_prod_layout_for(cfg: tq_config) -> tq_prod_layout:
    lay = tq_prod_layout()
    _abi.check("tq_prod_layout_for", _LIB.tq_prod_layout_for(ctypes.byref(cfg), ctypes.byref(lay)))
    return lay


def tq_prod_store(cfg: tq_config, cb, S: torch.Tensor, key: torch.Tensor, slot_mapping: torch.Tensor,
                  cache: torch.Tensor, num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
                  stream=None) -> None:
    """TurboQuant_prod keys: key [N, n_kv, d] f16/bf16, S fp32 [d, d] (row i =
    projection i), slot_mapping [N] int64, cache uint8 (the prod key cache)."""
    if S.dtype != torch.float32:
        raise ValueError("S must be float32")
    lay = tq_prod_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_prod_store", _LIB.tq_prod_store(
        ctypes.byref(cfg), _cb(cb), _ptr(S), _ptr(key), _DTYPES[key.dtype], key.shape[0], _ptr(slot_mapping),
        _ptr(cache), num_blocks, _ptr(dev_status), _stream(stream)))


def tq_prod_scores_workspace_size(cfg: tq_config, batch: int) -> int:
    return int(_LIB.tq_prod_scores_workspace_size(ctypes.byref(cfg), batch))


def tq_prod_scores(cfg: tq_config, cb, S: torch.Tensor, q: torch.Tensor, cache: torch.Tensor,
                   block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, scores: torch.Tensor,
                   workspace: torch.Tensor, scale: float = 0.0, num_blocks: int | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> None:
    """scores fp32 [B, n_q, max_seq_len]: scale * the unbiased estimate of <q, k_p>."""
    if S.dtype != torch.float32 or scores.dtype != torch.float32:
        raise ValueError("S and scores must be float32")
    lay = tq_prod_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_prod_scores", _LIB.tq_prod_scores(
        ctypes.byref(cfg), _cb(cb), _ptr(S), _ptr(q), _DTYPES[q.dtype], _ptr(cache), num_blocks,
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0], max_seq_len, float(scale),
        _ptr(scores), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status),
        _stream(stream)))


def tq_continue_workspace_size(cfg: tq_config, total_q: int, max_seq_len: int) -> int:
    return int(_LIB.tq_continue_workspace_size(ctypes.byref(cfg), total_q, max_seq_len))


def tq_continue(cfg: tq_config, cb, q: torch.Tensor, query_start: torch.Tensor, max_q_len: int,
                cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                out: torch.Tensor, workspace: torch.Tensor, scale: float = 0.0, num_blocks: int | None = None,
                dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Causal attention of continuation chunks: q [total_q, n_q, d], query_start
    int32 [batch + 1], seq_lens int32 [batch] (lengths with the chunk),
    block_table int32 [batch, stride], out [total_q, n_q, d]."""
    lay = tq_layout_for(cfg)
    if num_blocks is None:
        num_blocks = cache.numel() // lay.block_bytes
    _abi.check("tq_continue", _LIB.tq_continue(
        ctypes.byref(cfg), _cb(cb), _ptr(q), _DTYPES[q.dtype], _ptr(query_start), seq_lens.shape[0], q.shape[0],
        max_q_len, _ptr(cache), num_blocks, _ptr(block_table), block_table.shape[1], _ptr(seq_lens), max_seq_len,
        float(scale), _ptr(out), _DTYPES[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _stream(stream)))


# ---- 8-bit cache with a scale per block and head (e4m3_blk, int8_blk) ----------

def tq_b8_layout_for(cfg: tq_config) -> tq_b8_layout:
    lay = tq_b8_layout()
    _abi.check("tq_b8_layout_for", _LIB.tq_b8_layout_for(ctypes.byref(cfg), ctypes.byref(lay)))
    return lay


_B8_TYPES = (torch.float16, torch.bfloat16)


def _b8_rows(name: str, t: torch.Tensor, heads: int, d: int) -> int:
    """Checks a [rows, heads, d] tensor whose rows may be a stride apart (a slice
    of a fused projection's output); returns that stride in elements."""
    if t.dtype not in _B8_TYPES or t.dim() != 3 or t.shape[1:] != (heads, d):
        raise ValueError(f"{name} must be [rows, {heads}, {d}] float16 or bfloat16, got {tuple(t.shape)} {t.dtype}")
    s0, s1, s2 = t.stride()
    if t.shape[0] == 0:
        return heads * d
    if s2 != 1 or (s1 != d and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {(s0, s1, s2)}")
    if t.shape[0] == 1:
        return heads * d
    if s0 < heads * d:
        raise ValueError(f"{name}: the rows must not overlap, got strides {(s0, s1, s2)}")
    return s0


def _b8_common(cfg: tq_config, cache: torch.Tensor, num_blocks, block_table: torch.Tensor, seq_lens: torch.Tensor,
               others, stream, block_bytes=None) -> tuple:
    """What every call on the cache (8 or 16 bits) has in common: index tensors, one
    device, the current one (the library launches there), and the cache's size.
    Returns (num_blocks, row length of the table, raw stream)."""
    if cache.dtype != torch.uint8 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 tensor")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 matrix [batch, blocks]")
    if seq_lens.dtype != torch.int32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 vector")
    rows, width = block_table.shape
    if rows < seq_lens.shape[0]:
        raise ValueError("block_table has fewer rows than seq_lens has entries")
    dev = cache.get_device()
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    for t in (block_table, seq_lens, *others):
        if t is not None and t.get_device() != dev:
            raise ValueError("the tensors must be on one CUDA device")
    if dev != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)   # what torch.cuda.current_stream() wraps
    elif stream.device_index != dev:
        raise ValueError("the stream must be one of the tensors' device")
    else:
        raw = stream.cuda_stream
    have = cache.numel() // (block_bytes or _b8_block_bytes)(cfg.preset, cfg.head_dim, cfg.block_size, cfg.num_kv_heads)
    if num_blocks is None:
        num_blocks = have
    elif num_blocks > have:
        raise ValueError(f"cache holds {have} blocks, not {num_blocks}")
    return num_blocks, width, raw


@functools.lru_cache(maxsize=256)
def _b8_block_bytes(preset: int, head_dim: int, block_size: int, num_kv_heads: int) -> int:
    return tq_b8_layout_for(make_config(preset, num_kv_heads, num_kv_heads, head_dim, block_size)).block_bytes


def _b8_starts(query_start: torch.Tensor, seq_lens: torch.Tensor) -> None:
    if query_start.dtype != torch.int32 or not query_start.is_contiguous() or query_start.numel() != seq_lens.shape[0] + 1:
        raise ValueError("query_start must be a contiguous int32 vector of batch + 1 entries")


def _b8_out(name: str, t: torch.Tensor, shape) -> int:
    if t.dtype not in _DTYPES or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float16, bfloat16 or float32 tensor of shape {tuple(shape)}")
    return _DTYPES[t.dtype]


def _b8_workspace(t: torch.Tensor) -> int:
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


def _b8_status(t):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor")
    return t.data_ptr()


def tq_b8_store(cfg: tq_config, key: torch.Tensor, value: torch.Tensor, query_start: torch.Tensor, max_q_len: int,
                cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, num_blocks: int | None = None,
                dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Quantise chunks of new tokens into the cache: key, value [total_q, n_kv, d]
    f16/bf16 (rows may be a stride apart); rows query_start[b] ..
    query_start[b + 1] - 1 become the last positions of sequence b; seq_lens
    [batch] int32 are the lengths with the chunk."""
    ks = _b8_rows("key", key, cfg.num_kv_heads, cfg.head_dim)
    vs = _b8_rows("value", value, cfg.num_kv_heads, cfg.head_dim)
    if key.dtype != value.dtype or key.shape[0] != value.shape[0]:
        raise ValueError("key and value must have one dtype and one number of rows")
    _b8_starts(query_start, seq_lens)
    nb, width, raw = _b8_common(cfg, cache, num_blocks, block_table, seq_lens, (key, value, query_start, dev_status), stream)
    st = _LIB.tq_b8_store(cfg, key.data_ptr(), ks, value.data_ptr(), vs, _DTYPES[key.dtype], query_start.data_ptr(),
                          seq_lens.shape[0], key.shape[0], max_q_len, cache.data_ptr(), nb, block_table.data_ptr(), width,
                          seq_lens.data_ptr(), _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_b8_store", st)


def tq_b8_dequant(cfg: tq_config, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  max_seq_len: int, key_out: torch.Tensor, value_out: torch.Tensor, num_blocks: int | None = None,
                  dev_status: torch.Tensor | None = None, stream=None) -> None:
    """key_out, value_out [B, max_seq_len, n_kv, d] (f16, bf16 or f32), written in full."""
    shape = (seq_lens.shape[0], max_seq_len, cfg.num_kv_heads, cfg.head_dim)
    out_type = _b8_out("key_out", key_out, shape)
    if _b8_out("value_out", value_out, shape) != out_type:
        raise ValueError("key_out and value_out must have the same dtype")
    nb, width, raw = _b8_common(cfg, cache, num_blocks, block_table, seq_lens, (key_out, value_out, dev_status), stream)
    st = _LIB.tq_b8_dequant(cfg, cache.data_ptr(), nb, block_table.data_ptr(), width, seq_lens.data_ptr(), shape[0],
                            max_seq_len, key_out.data_ptr(), value_out.data_ptr(), out_type, _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_b8_dequant", st)


def tq_b8_decode_workspace_size(cfg: tq_config, batch: int, max_seq_len: int) -> int:
    return int(_LIB.tq_b8_decode_workspace_size(ctypes.byref(cfg), batch, max_seq_len))


def tq_b8_decode(cfg: tq_config, q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, max_seq_len: int, out: torch.Tensor, workspace: torch.Tensor,
                 scale: float = 0.0, num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
                 stream=None) -> None:
    """q [B, n_q, d] f16/bf16 (rows may be a stride apart); out [B, n_q, d]; seq_lens [B] int32."""
    qs = _b8_rows("q", q, cfg.num_q_heads, cfg.head_dim)
    out_type = _b8_out("out", out, q.shape)
    if q.shape[0] != seq_lens.shape[0]:
        raise ValueError("q must have one row per sequence")
    nb, width, raw = _b8_common(cfg, cache, num_blocks, block_table, seq_lens, (q, out, workspace, dev_status), stream)
    st = _LIB.tq_b8_decode(cfg, q.data_ptr(), qs, _DTYPES[q.dtype], cache.data_ptr(), nb, block_table.data_ptr(), width,
                           seq_lens.data_ptr(), q.shape[0], max_seq_len, scale, out.data_ptr(), out_type,
                           workspace.data_ptr(), _b8_workspace(workspace), _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_b8_decode", st)


def tq_b8_continue_workspace_size(cfg: tq_config, batch: int, total_q: int, max_q_len: int, max_seq_len: int) -> int:
    return int(_LIB.tq_b8_continue_workspace_size(ctypes.byref(cfg), batch, total_q, max_q_len, max_seq_len))


def tq_b8_continue(cfg: tq_config, q: torch.Tensor, query_start: torch.Tensor, max_q_len: int, cache: torch.Tensor,
                   block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, out: torch.Tensor,
                   workspace: torch.Tensor, scale: float = 0.0, num_blocks: int | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Causal attention of chunks whose keys and values are stored: q [total_q,
    n_q, d] f16/bf16 (rows may be a stride apart), query_start int32 [batch + 1],
    seq_lens int32 [batch] (lengths with the chunk), out [total_q, n_q, d]; rows
    of out from query_start[batch] on are left as they are."""
    qs = _b8_rows("q", q, cfg.num_q_heads, cfg.head_dim)
    out_type = _b8_out("out", out, q.shape)
    _b8_starts(query_start, seq_lens)
    nb, width, raw = _b8_common(cfg, cache, num_blocks, block_table, seq_lens, (q, query_start, out, workspace, dev_status), stream)
    st = _LIB.tq_b8_continue(cfg, q.data_ptr(), qs, _DTYPES[q.dtype], query_start.data_ptr(), seq_lens.shape[0], q.shape[0],
                             max_q_len, cache.data_ptr(), nb, block_table.data_ptr(), width, seq_lens.data_ptr(),
                             max_seq_len, scale, out.data_ptr(), out_type, workspace.data_ptr(),
                             _b8_workspace(workspace), _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_b8_continue", st)


# ---- 16-bit cache, with the position rotation on the way in (kv_bf16, kv_fp16) --

def tq_kv16_layout_for(cfg: tq_config) -> tq_kv16_layout:
    lay = tq_kv16_layout()
    _abi.check("tq_kv16_layout_for", _LIB.tq_kv16_layout_for(ctypes.byref(cfg), ctypes.byref(lay)))
    return lay


@functools.lru_cache(maxsize=256)
def _kv16_block_bytes(preset: int, head_dim: int, block_size: int, num_kv_heads: int) -> int:
    return tq_kv16_layout_for(make_config(preset, num_kv_heads, num_kv_heads, head_dim, block_size)).block_bytes


_KV16_TYPES = {TQ_PRESET_KV_BF16: torch.bfloat16, TQ_PRESET_KV_F16: torch.float16}


def _kv16_rows(name: str, t: torch.Tensor, kind: torch.dtype, heads: int, d: int) -> tuple:
    """As _b8_rows, of the cache's own type (which it looks at first: the usual call is over at once). Returns the
    number of rows and their stride."""
    if t.dtype is not kind:
        raise ValueError(f"{name} must have the cache's type, got {t.dtype}")
    shape = t.shape
    if len(shape) == 3:
        rows, have, last = shape
        s0, s1, s2 = t.stride()
        if have == heads and last == d and s2 == 1 and s1 == d and s0 >= heads * d and s0 % 8 == 0:
            return rows, s0
    return shape[0] if len(shape) else 0, _b8_rows(name, t, heads, d)


def _kv16_common(cfg: tq_config, cache: torch.Tensor, num_blocks, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 others: tuple, stream) -> tuple:
    """As _b8_common for the 16-bit cache: what a usual call has is checked at once, anything else goes there."""
    if (cache.dtype is torch.uint8 and block_table.dtype is torch.int32 and seq_lens.dtype is torch.int32 and num_blocks is None
            and stream is None and cache.is_contiguous() and block_table.is_contiguous() and block_table.dim() == 2
            and seq_lens.is_contiguous() and seq_lens.dim() == 1):
        rows, width = block_table.shape
        dev = cache.get_device()
        if rows >= seq_lens.shape[0] and dev >= 0 and dev == torch._C._cuda_getDevice():   # what current_device() asks
            for t in (block_table, seq_lens, *others):
                if t is not None and t.get_device() != dev:
                    break
            else:
                return (cache.numel() // _kv16_block_bytes(cfg.preset, cfg.head_dim, cfg.block_size, cfg.num_kv_heads), width,
                        torch._C._cuda_getCurrentRawStream(dev))
    return _b8_common(cfg, cache, num_blocks, block_table, seq_lens, others, stream, _kv16_block_bytes)


@functools.lru_cache(maxsize=None)
def _kv16_fn(name: str):
    return getattr(_LIB, name)


def _kv16_type(cfg: tq_config) -> torch.dtype:
    kind = _KV16_TYPES.get(cfg.preset)
    if kind is None:
        raise ValueError("the config must be of kv_bf16 or kv_fp16")
    return kind


def tq_kv16_append(cfg: tq_config, key: torch.Tensor, value: torch.Tensor, query_start: torch.Tensor, cache: torch.Tensor,
                   block_table: torch.Tensor, seq_lens: torch.Tensor, cos_sin: torch.Tensor | None = None,
                   style: str = "halves", q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                   num_blocks: int | None = None, dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Rotate chunks of new tokens by their positions and write them into the
    cache: key, value [total_q, n_kv, d], rows query_start[b] .. query_start[b + 1]
    - 1 become the last positions of sequence b, seq_lens [batch] int32 are the
    lengths with the chunk. cos_sin [positions, rot_dim] float32 (rot_dim / 2
    cosines, then as many sines) pairs a head's first rot_dim coordinates as
    `style` says, "halves" or "pairs"; None: no rotation. q [total_q, n_q, d] is
    rotated into q_out (which may be q). Rows may be a stride apart."""
    kind, heads, d = _kv16_type(cfg), cfg.num_kv_heads, cfg.head_dim
    rows, ks = _kv16_rows("key", key, kind, heads, d)
    same, vs = _kv16_rows("value", value, kind, heads, d)
    if same != rows:
        raise ValueError("key and value must have one number of rows")
    qs = os_ = rot = positions = 0
    q_at = out_at = angles = None
    if q is not None or q_out is not None:
        if q is None or q_out is None:
            raise ValueError("q and q_out must be given together")
        heads = cfg.num_q_heads
        same, qs = _kv16_rows("q", q, kind, heads, d)
        those, os_ = _kv16_rows("q_out", q_out, kind, heads, d)
        if same != rows or those != rows:
            raise ValueError("q, q_out and key must have one number of rows")
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    if cos_sin is not None:
        shape = cos_sin.shape
        if cos_sin.dtype != torch.float32 or len(shape) != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 matrix [positions, rot_dim]")
        positions, rot = shape
        if rot == 0:
            raise ValueError("cos_sin must have columns (None: no rotation)")
        angles = cos_sin.data_ptr()
    how = ROPE_STYLES.get(style)
    if how is None:
        raise ValueError(f"style must be one of {sorted(ROPE_STYLES)}, got {style!r}")
    _b8_starts(query_start, seq_lens)
    nb, width, raw = _kv16_common(cfg, cache, num_blocks, block_table, seq_lens,
                                  (key, value, query_start, q, q_out, cos_sin, dev_status), stream)
    st = _kv16_fn("tq_kv16_append")(cfg, key.data_ptr(), ks, value.data_ptr(), vs, q_at, qs, out_at, os_, angles, rot, positions, how,
                             query_start.data_ptr(), seq_lens.shape[0], rows, cache.data_ptr(), nb, block_table.data_ptr(), width,
                             seq_lens.data_ptr(), _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_kv16_append", st)


def tq_kv16_decode_workspace_size(cfg: tq_config, batch: int, max_seq_len: int) -> int:
    return int(_LIB.tq_kv16_decode_workspace_size(ctypes.byref(cfg), batch, max_seq_len))


def tq_kv16_decode(cfg: tq_config, q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                   seq_lens: torch.Tensor, max_seq_len: int, out: torch.Tensor, workspace: torch.Tensor,
                   scale: float = 0.0, num_blocks: int | None = None, dev_status: torch.Tensor | None = None,
                   stream=None) -> None:
    """q [B, n_q, d] of the cache's type (rows may be a stride apart); out [B, n_q, d]; seq_lens [B] int32."""
    rows, qs = _kv16_rows("q", q, _kv16_type(cfg), cfg.num_q_heads, cfg.head_dim)
    out_type = _b8_out("out", out, q.shape)
    if rows != seq_lens.shape[0]:
        raise ValueError("q must have one row per sequence")
    nb, width, raw = _kv16_common(cfg, cache, num_blocks, block_table, seq_lens, (q, out, workspace, dev_status), stream)
    st = _kv16_fn("tq_kv16_decode")(cfg, q.data_ptr(), qs, cache.data_ptr(), nb, block_table.data_ptr(), width, seq_lens.data_ptr(),
                             rows, max_seq_len, scale, out.data_ptr(), out_type, workspace.data_ptr(),
                             _b8_workspace(workspace), _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_kv16_decode", st)


def tq_kv16_continue_workspace_size(cfg: tq_config, batch: int, total_q: int, max_q_len: int, max_seq_len: int) -> int:
    return int(_LIB.tq_kv16_continue_workspace_size(ctypes.byref(cfg), batch, total_q, max_q_len, max_seq_len))


def tq_kv16_continue(cfg: tq_config, q: torch.Tensor, query_start: torch.Tensor, max_q_len: int, cache: torch.Tensor,
                     block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, out: torch.Tensor,
                     workspace: torch.Tensor, scale: float = 0.0, num_blocks: int | None = None,
                     dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Causal attention of chunks whose keys and values are stored: q [total_q,
    n_q, d] of the cache's type (rows may be a stride apart), query_start int32
    [batch + 1], seq_lens int32 [batch] (lengths with the chunk), out [total_q,
    n_q, d]; rows of out from query_start[batch] on are left as they are."""
    rows, qs = _kv16_rows("q", q, _kv16_type(cfg), cfg.num_q_heads, cfg.head_dim)
    out_type = _b8_out("out", out, q.shape)
    _b8_starts(query_start, seq_lens)
    nb, width, raw = _kv16_common(cfg, cache, num_blocks, block_table, seq_lens, (q, query_start, out, workspace, dev_status), stream)
    st = _kv16_fn("tq_kv16_continue")(cfg, q.data_ptr(), qs, query_start.data_ptr(), seq_lens.shape[0], rows, max_q_len,
                               cache.data_ptr(), nb, block_table.data_ptr(), width, seq_lens.data_ptr(), max_seq_len, scale,
                               out.data_ptr(), out_type, workspace.data_ptr(), _b8_workspace(workspace), _b8_status(dev_status), raw)
    if st:
        raise TQError("tq_kv16_continue", st)
