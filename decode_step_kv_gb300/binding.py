"""Thin Python binding of the C-ABI library (argument marshalling only).

Every function here forwards torch tensors' device pointers to the same-named
``extern "C"`` entry point of ``libfa_decode.so`` (declared in
``include/fa_decode.h``); all arithmetic runs in the CUDA kernels.  There is
no fallback: if the library cannot be built or loaded, the first call raises.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional

import torch

from . import _build

_lock = threading.Lock()
_lib = None

FA_STATUS_LEN_CLAMPED = 1
FA_STATUS_BAD_BLOCK = 2
FA_STATUS_WAIT_TIMEOUT = 4
FA_STATUS_POS_RANGE = 8
FA_STATUS_BAD_SLOT = 16


class FaDecodeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load (building first if needed) the CUDA library."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build_if_missing else _build.LIB
            lib = ctypes.CDLL(path)
            P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong,
                                    ctypes.c_float, ctypes.c_size_t)
            lib.fa_decode.argtypes = [P, P, P, P, P, P, i32, i32, i32, f32, P, P, i32, i32, i32,
                                      i32, P, sz, P]
            lib.fa_decode.restype = i32
            lib.fa_decode_noalloc.argtypes = [P, P, P, P, P, P, i32, i32, i32, f32, P, P, i32,
                                              i32, i32, i32, P]
            lib.fa_decode_noalloc.restype = i32
            lib.fa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
            lib.fa_decode_workspace_size.restype = sz
            lib.fa_quantize_v_int8.argtypes = [P, i64, i32, P, P, P]
            lib.fa_quantize_v_int8.restype = i32
            lib.fa_decode_batch_invariant.argtypes = [P, P, P, P, P, P, i32, i32, i32, f32, P,
                                                      P, i32, i32, i32, i32, i32, P, sz, P]
            lib.fa_decode_batch_invariant.restype = i32
            lib.fa_decode_batch_invariant_workspace_size.argtypes = [i32, i32, i32, i32, i32,
                                                                     i32]
            lib.fa_decode_batch_invariant_workspace_size.restype = sz
            lib.fa_decode_multi_batch_invariant.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32,
                                                            f32, P, P, i32, i32, i32, i32, i32, P,
                                                            sz, P]
            lib.fa_decode_multi_batch_invariant.restype = i32
            lib.fa_decode_multi_batch_invariant_workspace_size.argtypes = [i32] * 7
            lib.fa_decode_multi_batch_invariant_workspace_size.restype = sz
            lib.fa_decode_ring_batch_invariant.argtypes = [P, P, P, P, P, i32, i32, i32, f32, P,
                                                           P, i32, i32, i32, P, sz, P]
            lib.fa_decode_ring_batch_invariant.restype = i32
            lib.fa_decode_multi.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, f32, P, P, i32,
                                            i32, i32, i32, P, sz, P]
            lib.fa_decode_multi.restype = i32
            lib.fa_decode_multi_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
            lib.fa_decode_multi_workspace_size.restype = sz
            lib.fa_decode_ring.argtypes = [P, P, P, P, P, i32, i32, i32, f32, P, P, i32, i32, P,
                                           sz, P]
            lib.fa_decode_ring.restype = i32
            lib.fa_append_kv_ring.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, P]
            lib.fa_append_kv_ring.restype = i32
            lib.fa_decode_slots.argtypes = [P, P, P, P, P, P, i32, i32, i32, f32, P, P, i32, i32,
                                            i32, i32, P, sz, P]
            lib.fa_decode_slots.restype = i32
            lib.fa_append_kv_slots.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                               P]
            lib.fa_append_kv_slots.restype = i32
            lib.fa_append_kv.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, P]
            lib.fa_append_kv.restype = i32
            lib.fa_append_kv_int4.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                              i32, i32, P]
            lib.fa_append_kv_int4.restype = i32
            lib.fa_gather_kv_int4.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                              i32, i32, P]
            lib.fa_gather_kv_int4.restype = i32
            lib.fa_decode_int4.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, f32, P, P, P,
                                           i32, i32, i32, i32, P, sz, P]
            lib.fa_decode_int4.restype = i32
            lib.fa_decode_int4_workspace_size.argtypes = [i32] * 8
            lib.fa_decode_int4_workspace_size.restype = sz
            lib.fa_decode_weights.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, f32, P, P, P,
                                              i32, i32, i32, i32, P, sz, P]
            lib.fa_decode_weights.restype = i32
            lib.fa_decode_weights_workspace_size.argtypes = [i32] * 7
            lib.fa_decode_weights_workspace_size.restype = sz
            lib.fa_evict_kv.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                        i32, i32, i32, P]
            lib.fa_evict_kv.restype = i32
            lib.fa_gather_kv_debug.argtypes = [P, i32, P, i32, i32, i32, i32, i32, i32, P, P]
            lib.fa_gather_kv_debug.restype = i32
            lib.fa_decode_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), P]
            lib.fa_decode_device_status.restype = i32
            lib.fa_decode_profile_next.argtypes = [P, P]
            lib.fa_decode_profile_next.restype = i32
            lib.fa_selftest_wait_timeout.argtypes = [P]
            lib.fa_selftest_wait_timeout.restype = i32
            lib.fa_decode_last_error.argtypes = []
            lib.fa_decode_last_error.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fa_decode takes device tensors")
    if not t.is_contiguous():
        raise ValueError("fa_decode takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int):
    if rc != 0:
        raise FaDecodeError(rc, load().fa_decode_last_error().decode())


def fa_decode_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                             max_kv_len: int, num_sms: int = 0) -> int:
    return int(load().fa_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                               max_kv_len, num_sms))


def fa_decode(q, k_cache, v_cache, v_scales, block_table, seq_lens, n_q_heads, n_kv_heads,
              head_dim, scale, window, out, *, batch=None, page_size=16,
              max_blocks_per_seq=None, num_blocks=None, workspace=None, stream=None):
    """One decode step: out[b,h] = softmax(scale q.K^T) V over the attended range.

    Layouts and rules are those of ``fa_decode`` in include/fa_decode.h.
    `batch` defaults to q.shape[0]; `max_blocks_per_seq` to the block table's
    row length (paged) or k_cache.shape[2] (contiguous); `num_blocks` to
    k_cache.shape[0] (paged).
    """
    if batch is None:
        batch = q.shape[0]
    if max_blocks_per_seq is None:
        max_blocks_per_seq = block_table.shape[1] if block_table is not None else k_cache.shape[2]
    if num_blocks is None:
        num_blocks = k_cache.shape[0] if block_table is not None else 0
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales),
                          _ptr(block_table), _ptr(seq_lens), int(n_q_heads), int(n_kv_heads),
                          int(head_dim), float(scale), _ptr(window), _ptr(out), int(batch),
                          int(page_size), int(max_blocks_per_seq), int(num_blocks),
                          _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_decode_batch_invariant(q, k_cache, v_cache, v_scales, block_table, seq_lens, n_q_heads,
                              n_kv_heads, head_dim, scale, window, out, *, split_tokens=512,
                              batch=None, page_size=16, max_blocks_per_seq=None, num_blocks=None,
                              workspace=None, stream=None):
    """fa_decode with splits of `split_tokens` keys fixed per sequence, so a
    sequence's output is the same bytes whatever else is in the batch.
    Arguments as ``fa_decode``; the workspace is sized by
    ``fa_decode_batch_invariant_workspace_size``."""
    if batch is None:
        batch = q.shape[0]
    if max_blocks_per_seq is None:
        max_blocks_per_seq = block_table.shape[1] if block_table is not None else k_cache.shape[2]
    if num_blocks is None:
        num_blocks = k_cache.shape[0] if block_table is not None else 0
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode_batch_invariant(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales), _ptr(block_table),
        _ptr(seq_lens), int(n_q_heads), int(n_kv_heads), int(head_dim), float(scale),
        _ptr(window), _ptr(out), int(batch), int(page_size), int(max_blocks_per_seq),
        int(num_blocks), int(split_tokens), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_decode_batch_invariant_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_kv_len,
                                             split_tokens=512) -> int:
    return int(load().fa_decode_batch_invariant_workspace_size(
        batch, n_q_heads, n_kv_heads, head_dim, max_kv_len, split_tokens))


def fa_decode_multi_batch_invariant(q, k_cache, v_cache, v_scales, block_table, seq_lens,
                                    n_q_heads, n_kv_heads, head_dim, scale, window, out, *,
                                    split_tokens=512, page_size=16, max_blocks_per_seq=None,
                                    num_blocks=None, workspace=None, stream=None):
    """fa_decode_multi with the batch-invariant plan (fixed splits per sequence)."""
    batch, tq = q.shape[0], q.shape[1]
    if max_blocks_per_seq is None:
        max_blocks_per_seq = block_table.shape[1] if block_table is not None else k_cache.shape[2]
    if num_blocks is None:
        num_blocks = k_cache.shape[0] if block_table is not None else 0
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode_multi_batch_invariant(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales), _ptr(block_table),
        _ptr(seq_lens), int(tq), int(n_q_heads), int(n_kv_heads), int(head_dim), float(scale),
        _ptr(window), _ptr(out), int(batch), int(page_size), int(max_blocks_per_seq),
        int(num_blocks), int(split_tokens), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_decode_multi_batch_invariant_workspace_size(batch, n_queries, n_q_heads, n_kv_heads,
                                                   head_dim, max_kv_len, split_tokens=512) -> int:
    return int(load().fa_decode_multi_batch_invariant_workspace_size(
        batch, n_queries, n_q_heads, n_kv_heads, head_dim, max_kv_len, split_tokens))


def fa_decode_ring_batch_invariant(q, k_cache, v_cache, v_scales, seq_lens, n_q_heads,
                                   n_kv_heads, head_dim, scale, window, out, *, split_tokens=512,
                                   workspace=None, stream=None):
    """fa_decode_ring with the batch-invariant plan (fixed splits per sequence)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode_ring_batch_invariant(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales), _ptr(seq_lens), int(n_q_heads),
        int(n_kv_heads), int(head_dim), float(scale), _ptr(window), _ptr(out), int(q.shape[0]),
        int(k_cache.shape[2]), int(split_tokens), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_decode_multi(q, k_cache, v_cache, v_scales, block_table, seq_lens, n_q_heads, n_kv_heads,
                    head_dim, scale, window, out, *, page_size=16, max_blocks_per_seq=None,
                    num_blocks=None, workspace=None, stream=None):
    """Multi-query decode: q [B, Tq, Hq, D] = each sequence's last Tq tokens,
    query j attending keys up to its own position; out [B, Tq, Hq, D]."""
    batch, tq = q.shape[0], q.shape[1]
    if max_blocks_per_seq is None:
        max_blocks_per_seq = block_table.shape[1] if block_table is not None else k_cache.shape[2]
    if num_blocks is None:
        num_blocks = k_cache.shape[0] if block_table is not None else 0
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode_multi(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales),
                                _ptr(block_table), _ptr(seq_lens), int(tq), int(n_q_heads),
                                int(n_kv_heads), int(head_dim), float(scale), _ptr(window),
                                _ptr(out), int(batch), int(page_size), int(max_blocks_per_seq),
                                int(num_blocks), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_decode_multi_workspace_size(batch, n_queries, n_q_heads, n_kv_heads, head_dim, max_kv_len,
                                   num_sms=0) -> int:
    return int(load().fa_decode_multi_workspace_size(batch, n_queries, n_q_heads, n_kv_heads,
                                                     head_dim, max_kv_len, num_sms))


def fa_decode_ring(q, k_cache, v_cache, v_scales, seq_lens, n_q_heads, n_kv_heads, head_dim,
                   scale, window, out, *, workspace=None, stream=None):
    """Decode over a ring cache [B, Hkv, capacity, D]: token t at row t % capacity,
    seq_lens = tokens seen (may exceed capacity)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode_ring(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales),
                               _ptr(seq_lens), int(n_q_heads), int(n_kv_heads), int(head_dim),
                               float(scale), _ptr(window), _ptr(out), int(q.shape[0]),
                               int(k_cache.shape[2]), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_append_kv_ring(k_new, v_new, k_cache, v_cache, v_scales, positions, *, stream=None):
    """Write this step's K / V rows into a ring cache at row position % capacity."""
    rc = load().fa_append_kv_ring(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(v_scales), _ptr(positions), int(k_new.shape[0]),
                                  int(k_new.shape[1]), int(k_new.shape[2]),
                                  int(k_cache.shape[2]), _stream(stream))
    _check(rc)


def fa_decode_slots(q, k_cache, v_cache, v_scales, slot_ids, seq_lens, n_q_heads, n_kv_heads,
                    head_dim, scale, window, out, *, ring=False, workspace=None, stream=None):
    """Decode where row b reads slot slot_ids[b] of a pool [n_slots, Hkv, capacity, D]
    of contiguous (ring=False) or ring (ring=True) caches."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_decode_slots(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales),
                                _ptr(slot_ids), _ptr(seq_lens), int(n_q_heads), int(n_kv_heads),
                                int(head_dim), float(scale), _ptr(window), _ptr(out),
                                int(q.shape[0]), int(k_cache.shape[0]), int(k_cache.shape[2]),
                                int(bool(ring)), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def fa_append_kv_slots(k_new, v_new, k_cache, v_cache, v_scales, slot_ids, positions, *,
                       ring=False, stream=None):
    """Write row b's K / V into slot slot_ids[b] of a pool [n_slots, Hkv, capacity, D]
    at token positions[b] (row positions[b] % capacity for a ring)."""
    rc = load().fa_append_kv_slots(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(v_scales), _ptr(slot_ids), _ptr(positions),
                                   int(k_new.shape[0]), int(k_new.shape[1]), int(k_new.shape[2]),
                                   int(k_cache.shape[0]), int(k_cache.shape[2]), int(bool(ring)),
                                   _stream(stream))
    _check(rc)


def fa_decode_noalloc(q, k_cache, v_cache, v_scales, block_table, seq_lens, n_q_heads,
                      n_kv_heads, head_dim, scale, window, out, *, batch=None, page_size=16,
                      max_blocks_per_seq=None, num_blocks=None, stream=None):
    """fa_decode without a workspace argument, for callers that cannot allocate.

    The scratch is a fixed array inside the library (FA_NOALLOC_SCRATCH_BYTES);
    sizes that need more raise FaDecodeError.  Calls that overlap on the GPU
    share that array and race, so keep them on one stream.
    """
    if batch is None:
        batch = q.shape[0]
    if max_blocks_per_seq is None:
        max_blocks_per_seq = block_table.shape[1] if block_table is not None else k_cache.shape[2]
    if num_blocks is None:
        num_blocks = k_cache.shape[0] if block_table is not None else 0
    rc = load().fa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scales),
                                  _ptr(block_table), _ptr(seq_lens), int(n_q_heads),
                                  int(n_kv_heads), int(head_dim), float(scale), _ptr(window),
                                  _ptr(out), int(batch), int(page_size),
                                  int(max_blocks_per_seq), int(num_blocks), _stream(stream))
    _check(rc)


def fa_quantize_v_int8(x, codes, scales, *, stream=None):
    """Pack fp32 x [..., D] into int8 codes [..., D] and fp16 scales [..., D/32]."""
    D = x.shape[-1]
    rc = load().fa_quantize_v_int8(_ptr(x), x.numel() // D, D, _ptr(codes), _ptr(scales),
                                   _stream(stream))
    _check(rc)


def fa_append_kv(k_new, v_new, k_cache, v_cache, v_scales, block_table, positions, *,
                 n_kv_heads, head_dim, page_size=16, max_blocks_per_seq=None, num_blocks=None,
                 stream=None):
    """Write this step's K / V rows ([B, Hkv, D] fp32) into the cache at `positions`."""
    batch = k_new.shape[0]
    if max_blocks_per_seq is None:
        max_blocks_per_seq = block_table.shape[1] if block_table is not None else k_cache.shape[2]
    if num_blocks is None:
        num_blocks = k_cache.shape[0] if block_table is not None else 0
    rc = load().fa_append_kv(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                             _ptr(v_scales), _ptr(block_table), _ptr(positions), int(batch),
                             int(n_kv_heads), int(head_dim), int(page_size),
                             int(max_blocks_per_seq), int(num_blocks), _stream(stream))
    _check(rc)


def _take(name, t, dtype, shape, dev):
    """Device pointer (None for None) of a contiguous tensor of `dtype` and
    `shape` (None: any) on device `dev`."""
    if t is None:
        return None
    if (t.dtype is dtype and (shape is None or t.shape == shape) and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _device():
    """The current CUDA device (None without one: no tensor is on it)."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None


def _cache_dims(name, k, block_table, batch):
    """(kv heads, page_size, max_blocks_per_seq, num_blocks, row shape, row elements) of a
    cache [num_blocks, Hkv, page, ...] (paged) or [batch, Hkv, capacity, ...]."""
    shape = k.shape
    if len(shape) != 4:
        raise ValueError(f"{name}: caches are [blocks or batch, kv heads, page or capacity, row]")
    n, hkv, page, width = shape
    if block_table is None:
        if n != batch:
            raise ValueError(f"{name}: a contiguous cache holds {n} sequences, "
                             f"the call has {batch}")
        return hkv, 16, page, 0, (n, hkv, page), width
    table = block_table.shape
    if len(table) != 2 or table[0] != batch:
        raise ValueError(f"{name}: block_table must be [batch, max_blocks_per_seq]")
    return hkv, page, table[1], n, (n, hkv, page), width


def _stream_ptr(stream, dev):
    return (torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def _workspace(t, dev):
    """Pointer and bytes of a workspace of any type."""
    if t is None:
        return None, 0
    return _take("workspace", t, t.dtype, None, dev), t.numel() * t.element_size()


def _int4_cache(name, k_codes, k_scales, v_codes, v_scales, block_table, batch, dev):
    """Pointers and sizes of a 4-bit cache: (pointers, table, kv heads, page,
    max_blocks, num_blocks, rows, head_dim)."""
    hkv, page, blocks, total, rows, half = _cache_dims(name, k_codes, block_table, batch)
    scales = (*rows, half // 16)
    ptrs = (_take("k_codes", k_codes, torch.uint8, None, dev),
            _take("k_scales", k_scales, torch.float16, scales, dev),
            _take("v_codes", v_codes, torch.uint8, (*rows, half), dev),
            _take("v_scales", v_scales, torch.float16, scales, dev))
    return (ptrs, _take("block_table", block_table, torch.int32, None, dev), hkv, page, blocks,
            total, rows, 2 * half)


def fa_append_kv_int4(k_new, v_new, k_codes, k_scales, v_codes, v_scales, block_table, positions,
                      *, n_new=None, stream=None):
    """Write rows k_new / v_new [B, T, Hkv, D] fp32 into a 4-bit cache, sequence b's
    row i at token positions[b] + i; `n_new` [B] int32: only the first n_new[b] rows.

    codes: uint8 [blocks, Hkv, page, D/2] with a block_table, or [B, Hkv, capacity, D/2];
    scales: fp16 [..., D/32] beside them."""
    shape = k_new.shape
    B, T = shape[0], shape[1]
    dev = _device()
    c, bt, hkv, page, blocks, total, _, D = _int4_cache("fa_append_kv_int4", k_codes, k_scales,
                                                        v_codes, v_scales, block_table, B, dev)
    new = (B, T, hkv, D)
    _check(load().fa_append_kv_int4(
        _take("k_new", k_new, torch.float32, new, dev),
        _take("v_new", v_new, torch.float32, new, dev), *c, bt,
        _take("positions", positions, torch.int32, (B,), dev),
        _take("n_new", n_new, torch.int32, (B,), dev), B, T, hkv, D, page, blocks, total,
        _stream_ptr(stream, dev)))


def fa_gather_kv_int4(k_codes, k_scales, v_codes, v_scales, block_table, positions, k_out, v_out,
                      *, n_rows=None, stream=None):
    """Rows positions[b] + i of a 4-bit cache as fp16 k_out / v_out [B, T, Hkv, D];
    `n_rows` [B] int32: only the first n_rows[b] of them."""
    shape = k_out.shape
    B, T = shape[0], shape[1]
    dev = _device()
    c, bt, hkv, page, blocks, total, _, D = _int4_cache("fa_gather_kv_int4", k_codes, k_scales,
                                                        v_codes, v_scales, block_table, B, dev)
    to = (B, T, hkv, D)
    _check(load().fa_gather_kv_int4(
        *c, bt, _take("positions", positions, torch.int32, (B,), dev),
        _take("n_rows", n_rows, torch.int32, (B,), dev),
        _take("k_out", k_out, torch.float16, to, dev),
        _take("v_out", v_out, torch.float16, to, dev), B, T, hkv, D, page, blocks, total,
        _stream_ptr(stream, dev)))


def _queries(name, q, out, n_q_heads, head_dim, dev):
    """(batch, queries, q pointer, out pointer) of q and out, [B, Hq, D] or [B, Tq, Hq, D]."""
    shape = q.shape
    n = len(shape)
    if (n != 3 and n != 4) or shape[n - 2] != n_q_heads or shape[n - 1] != head_dim:
        raise ValueError(f"{name}: q must be [B, Hq, D] or [B, Tq, Hq, D]")
    return (shape[0], 1 if n == 3 else shape[1],
            _take("q", q, torch.float16, None, dev), _take("out", out, torch.float16, shape, dev))


def fa_decode_int4(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, n_q_heads,
                   n_kv_heads, head_dim, scale, window, out, *, acc=None, workspace=None,
                   stream=None):
    """Decode attention over a 4-bit cache: q, out fp16 [B, Hq, D] (one query per
    sequence) or [B, Tq, Hq, D] (each sequence's last Tq tokens, causal).  `acc`
    (fp32, one value per cache row) also gets every key's softmax weight added, as in
    ``fa_decode_weights``.  The workspace is ``alloc_workspace_int4``'s."""
    dev = _device()
    B, tq, qp, op = _queries("fa_decode_int4", q, out, n_q_heads, head_dim, dev)
    c, bt, hkv, page, blocks, total, rows, D = _int4_cache("fa_decode_int4", k_codes, k_scales,
                                                           v_codes, v_scales, block_table, B, dev)
    if hkv != n_kv_heads or D != head_dim:
        raise ValueError(f"fa_decode_int4: the cache holds {hkv} heads of {D}")
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().fa_decode_int4(
        qp, *c, bt, _take("seq_lens", seq_lens, torch.int32, (B,), dev), tq, n_q_heads, hkv, D,
        scale, _take("window", window, torch.int32, (B,), dev), op,
        _take("acc", acc, torch.float32, rows, dev), B, page, blocks, total, ws, ws_bytes,
        _stream_ptr(stream, dev)))


def fa_decode_int4_workspace_size(batch, n_queries, n_q_heads, n_kv_heads, head_dim, max_kv_len,
                                  with_weights=False, num_sms=0) -> int:
    return int(load().fa_decode_int4_workspace_size(batch, n_queries, n_q_heads, n_kv_heads,
                                                    head_dim, max_kv_len, int(with_weights),
                                                    num_sms))


def alloc_workspace_int4(batch, n_queries, n_q_heads, n_kv_heads, head_dim, max_kv_len, *,
                         weights=False, device="cuda"):
    """Device scratch for fa_decode_int4 (weights=True: for calls with acc too)."""
    n = fa_decode_int4_workspace_size(batch, n_queries, n_q_heads, n_kv_heads, head_dim,
                                      max_kv_len, weights)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def fa_decode_weights(q, k_cache, v_cache, v_scales, block_table, seq_lens, n_q_heads, n_kv_heads,
                      head_dim, scale, window, out, acc, *, workspace=None, stream=None):
    """``fa_decode_multi`` (q fp16 [B, Hq, D] or [B, Tq, Hq, D]) with fp16 out, which also
    adds every key's softmax weight, summed over the queries and the query heads of its
    KV head, to `acc` (fp32, one value per cache row: the cache's shape without D).
    The workspace is ``alloc_workspace_weights``'s."""
    dev = _device()
    hkv, page, blocks, total, rows, _ = _cache_dims("fa_decode_weights", k_cache, block_table,
                                                    q.shape[0])
    B, tq, qp, op = _queries("fa_decode_weights", q, out, n_q_heads, head_dim, dev)
    if hkv != n_kv_heads:
        raise ValueError(f"fa_decode_weights: the cache holds {hkv} heads")
    row = (*rows, head_dim)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().fa_decode_weights(
        qp, _take("k_cache", k_cache, torch.float16, row, dev),
        _take("v_cache", v_cache, torch.float16 if v_scales is None else torch.int8, row, dev),
        _take("v_scales", v_scales, torch.float16, (*rows, head_dim // 32), dev),
        _take("block_table", block_table, torch.int32, None, dev),
        _take("seq_lens", seq_lens, torch.int32, (B,), dev), tq, n_q_heads, hkv, head_dim, scale,
        _take("window", window, torch.int32, (B,), dev), op,
        _take("acc", acc, torch.float32, rows, dev), B, page, blocks, total, ws, ws_bytes,
        _stream_ptr(stream, dev)))


def fa_decode_weights_workspace_size(batch, n_queries, n_q_heads, n_kv_heads, head_dim, max_kv_len,
                                     num_sms=0) -> int:
    return int(load().fa_decode_weights_workspace_size(batch, n_queries, n_q_heads, n_kv_heads,
                                                       head_dim, max_kv_len, num_sms))


def alloc_workspace_weights(batch, n_queries, n_q_heads, n_kv_heads, head_dim, max_kv_len, *,
                            device="cuda"):
    """Device scratch for fa_decode_weights."""
    n = fa_decode_weights_workspace_size(batch, n_queries, n_q_heads, n_kv_heads, head_dim,
                                         max_kv_len)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def fa_evict_kv(k_cache, v_cache, acc, block_table, seq_lens, new_lens, *, budget, n_sink,
                n_recent, kept, k_scales=None, v_scales=None, stream=None):
    """Cut every sequence to `budget` tokens per KV head, in place: the first n_sink, the
    last n_recent, and the largest `acc` totals between them (ties: lowest index), moved in
    order to the front.  fp16 caches; with v_scales, int8 V; with both scales, 4-bit K and V
    (uint8 codes).  Writes new_lens [B] and kept [B, Hkv, budget] (int32)."""
    B = seq_lens.shape[0]
    dev = _device()
    hkv, page, blocks, total, rows, width = _cache_dims("fa_evict_kv", k_cache, block_table, B)
    int4 = k_scales is not None
    D = width * (2 if int4 else 1)
    scales = (*rows, D // 32)
    v_type = torch.uint8 if int4 else torch.float16 if v_scales is None else torch.int8
    _check(load().fa_evict_kv(
        _take("k_cache", k_cache, torch.uint8 if int4 else torch.float16, None, dev),
        _take("v_cache", v_cache, v_type, k_cache.shape, dev),
        _take("k_scales", k_scales, torch.float16, scales, dev),
        _take("v_scales", v_scales, torch.float16, scales, dev),
        _take("acc", acc, torch.float32, rows, dev),
        _take("block_table", block_table, torch.int32, None, dev),
        _take("seq_lens", seq_lens, torch.int32, (B,), dev),
        _take("new_lens", new_lens, torch.int32, (B,), dev),
        _take("kept", kept, torch.int32, (B, hkv, budget), dev), budget, n_sink, n_recent, B, hkv,
        D, page, blocks, total, _stream_ptr(stream, dev)))


def fa_gather_kv_debug(cache, row_bytes, block_table, b, n_kv_heads, page_size,
                       max_blocks_per_seq, num_blocks, n_tokens, dense, *, stream=None):
    rc = load().fa_gather_kv_debug(_ptr(cache), int(row_bytes), _ptr(block_table), int(b),
                                   int(n_kv_heads), int(page_size), int(max_blocks_per_seq),
                                   int(num_blocks), int(n_tokens), _ptr(dense), _stream(stream))
    _check(rc)


def fa_decode_profile_next(split_start=None, split_end=None):
    """Record torch.cuda.Event objects around the next call's split kernel.

    The events must already exist on the device (torch creates them lazily at
    their first record()); a zero handle raises.
    """
    a = None if split_start is None else ctypes.c_void_p(split_start.cuda_event)
    b = None if split_end is None else ctypes.c_void_p(split_end.cuda_event)
    if (split_start is not None and not a.value) or (split_end is not None and not b.value):
        raise ValueError("fa_decode_profile_next: event not created yet (record it once first)")
    _check(load().fa_decode_profile_next(a, b))


def fa_selftest_wait_timeout(*, stream=None):
    """Launch the bounded-wait self-test (about one second; sets FA_STATUS_WAIT_TIMEOUT)."""
    _check(load().fa_selftest_wait_timeout(_stream(stream)))


def fa_decode_device_status(*, stream=None) -> int:
    v = ctypes.c_uint(0)
    _check(load().fa_decode_device_status(ctypes.byref(v), _stream(stream)))
    return int(v.value)


def alloc_workspace(batch, n_q_heads, n_kv_heads, head_dim, max_kv_len, device="cuda"):
    """Device scratch for fa_decode (torch allocation: plumbing, not compute)."""
    n = fa_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_kv_len)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)
