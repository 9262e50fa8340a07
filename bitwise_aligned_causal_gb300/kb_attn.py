"""ctypes binding of libkb_attn.so (C ABI in include/kb_attn.h).

Argument marshalling only: every step of the attention runs in the library's
CUDA kernels.  The functions named like the C entry points take raw device
pointers; ``prefill`` / ``chunk`` / ``decode`` accept torch CUDA tensors
(PyTorch is used here only for device memory and streams).

Importing this module loads the library and raises ``ImportError`` when it
has not been built: there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import functools
import os

from . import shapes

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkb_attn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with bitwise_aligned_causal_gb300.build.build()")
_lib = ctypes.CDLL(LIB_PATH)

KB_OK = 0
KB_ERR_INVALID_ARG = 1
KB_ERR_UNSUPPORTED = 2
KB_ERR_CUDA = 3
KB_ERR_TIMEOUT = 4

_P = ctypes.c_void_p
_I = ctypes.c_int
_N = ctypes.POINTER(ctypes.c_longlong)
_SIGS = {
    "kb_attn_prefill": [_P, _P, _P, _P, _I, _I, _I, _I, _P],
    "kb_attn_chunk": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P],
    "kb_attn_decode": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P],
    "kb_attn_decode_paged": [_P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _P, _P],
    "kb_attn_chunk_paged": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _I, _I, _P],
    "kb_attn_chunk_varlen": [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _I, _I, _I, _P],
    "kb_attn_check_device_status": [_P],
    "kb_attn_debug_wait_timeout": [_I, _P],
    "kb_attn_chunk_cta_shape": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P],
    "kb_attn_prefill_lse": [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P],
    "kb_attn_prefill_seg": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P],
    "kb_attn_chunk_seg": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, ctypes.c_size_t, _P],
    "kb_attn_decode_seg": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, ctypes.c_size_t, _P],
    "kb_attn_seg_workspace_bytes": [_I, _I, _I, _I, _I],
    "kb_attn_decode_seg_static": [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P],
    "kb_attn_backward": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P],
    "kb_attn_rope_table": [_P, _I, _I, _P, _P],
    "kb_attn_rope": [_P, _N, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P],
    "kb_attn_append": [_P, _P, _P, _N, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _I, _I, _I,
                       _P],
    "kb_attn_block_boxes": [_P, _P, _I, _I, _I, _P, _I, _P, _I, _I, _I, _P],
    "kb_attn_select_blocks": [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _I, _I, _I, _P],
    "kb_attn_sparse_workspace_bytes": [_I, _I, _I, _I, _I],
    "kb_attn_sparse_chunk": [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _I, _I, _I, _P,
                             ctypes.c_size_t, _P],
    "kb_attn_sparse_prefill_lse": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, ctypes.c_size_t, _P],
    "kb_attn_sparse_decode": [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P, _I, _I, _I, _P],
    "kb_attn_sparse_backward_workspace_bytes": [_I, _I, _I, _I],
    "kb_attn_sparse_backward": [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, ctypes.c_size_t,
                                _P],
    "kb_status_string": [_I],
    "kb_contract_version": [],
    "kb_attn_last_cuda_error": [],
    "kb_attn_last_cuda_error_string": [],
}
for _name, _args in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = (ctypes.c_char_p if _name.endswith("string")
                  else ctypes.c_size_t if _name.endswith("_bytes") else ctypes.c_int)

EXPORTED = tuple(_SIGS)


class KBError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {kb_status_string(status)} (status {status})"
        if status == KB_ERR_CUDA:
            msg += f": {kb_attn_last_cuda_error_string()} (cudaError {kb_attn_last_cuda_error()})"
        super().__init__(msg)


def kb_status_string(status: int) -> str:
    return _lib.kb_status_string(int(status)).decode()


def kb_contract_version() -> int:
    return int(_lib.kb_contract_version())


def kb_attn_last_cuda_error() -> int:
    return int(_lib.kb_attn_last_cuda_error())


def kb_attn_last_cuda_error_string() -> str:
    return _lib.kb_attn_last_cuda_error_string().decode()


# ---------------------------------------------------------------- raw C entry points

def kb_attn_prefill(q, k, v, o, B, Hq, Hkv, S, stream=None) -> int:
    return _lib.kb_attn_prefill(q, k, v, o, B, Hq, Hkv, S, stream)


def kb_attn_chunk(q, k, v, o, B, Hq, Hkv, L, start, kv_cap, stream=None) -> int:
    return _lib.kb_attn_chunk(q, k, v, o, B, Hq, Hkv, L, start, kv_cap, stream)


def kb_attn_decode(q, k, v, o, B, Hq, Hkv, ctx_len, kv_cap, stream=None) -> int:
    return _lib.kb_attn_decode(q, k, v, o, B, Hq, Hkv, ctx_len, kv_cap, stream)


def kb_attn_decode_paged(q, k_pages, v_pages, o, B, Hq, Hkv, block_table, pages_per_seq, page_size, num_pages,
                         ctx_lens, stream=None) -> int:
    return _lib.kb_attn_decode_paged(q, k_pages, v_pages, o, B, Hq, Hkv, block_table, pages_per_seq, page_size,
                                     num_pages, ctx_lens, stream)


def kb_attn_chunk_paged(q, k_pages, v_pages, o, B, Hq, Hkv, L, start, block_table, pages_per_seq, page_size,
                        num_pages, stream=None) -> int:
    return _lib.kb_attn_chunk_paged(q, k_pages, v_pages, o, B, Hq, Hkv, L, start, block_table, pages_per_seq,
                                    page_size, num_pages, stream)


def kb_attn_chunk_varlen(q, k, v, o, B, Hq, Hkv, L_max, starts, lens, kv_cap, block_table, pages_per_seq,
                         page_size, num_pages, stream=None) -> int:
    return _lib.kb_attn_chunk_varlen(q, k, v, o, B, Hq, Hkv, L_max, starts, lens, kv_cap, block_table, pages_per_seq,
                                     page_size, num_pages, stream)


def kb_attn_chunk_cta_shape(q, k, v, o, B, Hq, Hkv, L, start, kv_cap, q_tiles_per_cta, stream=None) -> int:
    return _lib.kb_attn_chunk_cta_shape(q, k, v, o, B, Hq, Hkv, L, start, kv_cap, q_tiles_per_cta, stream)


def kb_attn_prefill_lse(q, k, v, o, lse, B, Hq, Hkv, S, stream=None) -> int:
    return _lib.kb_attn_prefill_lse(q, k, v, o, lse, B, Hq, Hkv, S, stream)


def kb_attn_backward(q, k, v, o, dout, lse, delta, dq, dk, dv, B, Hq, Hkv, S, stream=None) -> int:
    return _lib.kb_attn_backward(q, k, v, o, dout, lse, delta, dq, dk, dv, B, Hq, Hkv, S, stream)


def kb_attn_prefill_seg(q, k, v, o, B, Hq, Hkv, S, seg_tiles, stream=None) -> int:
    return _lib.kb_attn_prefill_seg(q, k, v, o, B, Hq, Hkv, S, seg_tiles, stream)


def kb_attn_chunk_seg(q, k, v, o, B, Hq, Hkv, L, start, kv_cap, seg_tiles, workspace, workspace_bytes,
                      stream=None) -> int:
    return _lib.kb_attn_chunk_seg(q, k, v, o, B, Hq, Hkv, L, start, kv_cap, seg_tiles, workspace, workspace_bytes,
                                  stream)


def kb_attn_decode_seg(q, k, v, o, B, Hq, Hkv, ctx_len, kv_cap, seg_tiles, workspace, workspace_bytes,
                       stream=None) -> int:
    return _lib.kb_attn_decode_seg(q, k, v, o, B, Hq, Hkv, ctx_len, kv_cap, seg_tiles, workspace, workspace_bytes,
                                   stream)


def kb_attn_decode_seg_static(q, k, v, o, B, Hq, Hkv, ctx_len, kv_cap, seg_tiles, stream=None) -> int:
    return _lib.kb_attn_decode_seg_static(q, k, v, o, B, Hq, Hkv, ctx_len, kv_cap, seg_tiles, stream)


def kb_attn_seg_workspace_bytes(B, Hq, L, start, seg_tiles) -> int:
    return int(_lib.kb_attn_seg_workspace_bytes(B, Hq, L, start, seg_tiles))


def kb_attn_rope_table(table, n_pos, rot_dim, inv_freq, stream=None) -> int:
    return _lib.kb_attn_rope_table(table, n_pos, rot_dim, inv_freq, stream)


def kb_attn_rope(x, strides, out, table, n_pos, rot_dim, interleaved, inverse, B, H, L, start, stream=None) -> int:
    return _lib.kb_attn_rope(x, strides, out, table, n_pos, rot_dim, interleaved, inverse, B, H, L, start, stream)


def kb_attn_append(q, k, v, strides, q_out, k_cache, v_cache, boxes, table, n_pos, rot_dim, interleaved, B, Hq, Hkv, L,
                   start, starts, lens, kv_cap, block_table, pages_per_seq, page_size, num_pages, stream=None) -> int:
    return _lib.kb_attn_append(q, k, v, strides, q_out, k_cache, v_cache, boxes, table, n_pos, rot_dim, interleaved, B,
                               Hq, Hkv, L, start, starts, lens, kv_cap, block_table, pages_per_seq, page_size,
                               num_pages, stream)


def kb_attn_block_boxes(k_cache, boxes, B, Hkv, kv_len, kv_lens, kv_cap, block_table, pages_per_seq, page_size,
                        num_pages, stream=None) -> int:
    return _lib.kb_attn_block_boxes(k_cache, boxes, B, Hkv, kv_len, kv_lens, kv_cap, block_table, pages_per_seq,
                                    page_size, num_pages, stream)


def kb_attn_select_blocks(q, boxes, blocks, B, Hq, Hkv, L, n_select, keep_first, keep_last, start, starts, lens,
                          n_blocks, block_table, pages_per_seq, page_size, num_pages, stream=None) -> int:
    return _lib.kb_attn_select_blocks(q, boxes, blocks, B, Hq, Hkv, L, n_select, keep_first, keep_last, start, starts,
                                      lens, n_blocks, block_table, pages_per_seq, page_size, num_pages, stream)


def kb_attn_sparse_workspace_bytes(B, Hkv, L, n_select, kv_cap) -> int:
    return int(_lib.kb_attn_sparse_workspace_bytes(B, Hkv, L, n_select, kv_cap))


def kb_attn_sparse_chunk(q, k, v, o, blocks, n_select, B, Hq, Hkv, L, start, starts, lens, kv_cap, block_table,
                         pages_per_seq, page_size, num_pages, workspace, workspace_bytes, stream=None) -> int:
    return _lib.kb_attn_sparse_chunk(q, k, v, o, blocks, n_select, B, Hq, Hkv, L, start, starts, lens, kv_cap,
                                     block_table, pages_per_seq, page_size, num_pages, workspace, workspace_bytes,
                                     stream)


def kb_attn_sparse_prefill_lse(q, k, v, o, lse, blocks, n_select, B, Hq, Hkv, S, workspace, workspace_bytes,
                               stream=None) -> int:
    return _lib.kb_attn_sparse_prefill_lse(q, k, v, o, lse, blocks, n_select, B, Hq, Hkv, S, workspace,
                                           workspace_bytes, stream)


def kb_attn_sparse_decode(q, k, v, o, blocks, n_select, B, Hq, Hkv, ctx_len, ctx_lens, kv_cap, block_table,
                          pages_per_seq, page_size, num_pages, stream=None) -> int:
    return _lib.kb_attn_sparse_decode(q, k, v, o, blocks, n_select, B, Hq, Hkv, ctx_len, ctx_lens, kv_cap, block_table,
                                      pages_per_seq, page_size, num_pages, stream)


def kb_attn_sparse_backward_workspace_bytes(B, Hkv, S, n_select) -> int:
    return int(_lib.kb_attn_sparse_backward_workspace_bytes(B, Hkv, S, n_select))


def kb_attn_sparse_backward(q, k, v, o, dout, lse, delta, blocks, n_select, dq, dk, dv, B, Hq, Hkv, S, workspace,
                            workspace_bytes, stream=None) -> int:
    return _lib.kb_attn_sparse_backward(q, k, v, o, dout, lse, delta, blocks, n_select, dq, dk, dv, B, Hq, Hkv, S,
                                        workspace, workspace_bytes, stream)


def kb_attn_check_device_status(stream=None) -> int:
    return _lib.kb_attn_check_device_status(stream)


def kb_attn_debug_wait_timeout(limit_us, stream=None) -> int:
    return _lib.kb_attn_debug_wait_timeout(limit_us, stream)


# ------------------------------------------------------------------ torch marshalling
#
# Every wrapper below checks each tensor's dtype, layout, device and full
# shape against the others (shapes.py) before the C call, so a caller's
# mistake raises here instead of becoming an out-of-bounds device access.
#
# Outputs are complete once the stream has run the kernels.  A bounded
# device-side wait that gave up, or a device-resident argument found out of
# range (a page index, a per-sequence length), leaves the affected rows
# unwritten and is reported only by check_device_status(), which also clears
# the library's error word; until that word is cleared, later calls on the
# device skip their work.  Pass check=True to call it after the launch.

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on_current_device(t, name):
    torch = _torch()
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{torch.cuda.current_device()}")


def _check(t, name, ndim=4):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions [batch, heads, seq, head_dim]")
    _on_current_device(t, name)


def _check_i32(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    _on_current_device(t, name)


def _check_f32(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    _on_current_device(t, name)


def _raise(status, where):
    if status != KB_OK:
        raise KBError(status, where)


def _out(q, out):
    o = _torch().empty_like(q) if out is None else out
    _check(o, "out")
    return o


def _finish(status, where, check, stream):
    _raise(status, where)
    if check:
        check_device_status(stream)


def prefill(q, k, v, out=None, stream=None, check=False):
    """Causal prefill: q [B,Hq,S,128], k/v [B,Hkv,S,128] -> o shaped like q."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, S = shapes.prefill(q.shape, k.shape, v.shape, None if out is None else out.shape)
    o = _out(q, out)
    _finish(kb_attn_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, S, _stream(stream)),
            "kb_attn_prefill", check, stream)
    return o


def chunk(q, k, v, start, out=None, stream=None, q_tiles_per_cta=None, check=False):
    """Chunked forward: q [B,Hq,L,128] at positions start.., k/v caches [B,Hkv,cap,128]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, L, cap = shapes.chunk(q.shape, k.shape, v.shape, int(start), None if out is None else out.shape)
    o = _out(q, out)
    if q_tiles_per_cta is None:
        st = kb_attn_chunk(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, L, int(start), cap,
                           _stream(stream))
    else:
        st = kb_attn_chunk_cta_shape(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, L,
                                     int(start), cap, int(q_tiles_per_cta), _stream(stream))
    _finish(st, "kb_attn_chunk", check, stream)
    return o


def decode(q, k, v, ctx_len, out=None, stream=None, check=False):
    """One-token decode: q [B,Hq,1,128] at position ctx_len-1, k/v caches [B,Hkv,cap,128]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, cap = shapes.decode(q.shape, k.shape, v.shape, int(ctx_len), None if out is None else out.shape)
    o = _out(q, out)
    _finish(kb_attn_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, int(ctx_len), cap,
                           _stream(stream)), "kb_attn_decode", check, stream)
    return o


def decode_paged(q, k_pages, v_pages, block_table, ctx_lens, out=None, stream=None, check=False):
    """Paged decode: q [B,Hq,1,128]; pools [num_pages,Hkv,page_size,128]; block_table int32 [B,pages_per_seq];
    ctx_lens int32 [B] (all on the device)."""
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _check(t, n)
    for t, n in ((block_table, "block_table"), (ctx_lens, "ctx_lens")):
        _check_i32(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, num_pages, page_size, pps = shapes.decode_paged(
        q.shape, k_pages.shape, v_pages.shape, block_table.shape, ctx_lens.shape, None if out is None else out.shape)
    o = _out(q, out)
    _finish(kb_attn_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), o.data_ptr(), B, Hq, Hkv,
                                 block_table.data_ptr(), pps, page_size, num_pages, ctx_lens.data_ptr(),
                                 _stream(stream)), "kb_attn_decode_paged", check, stream)
    return o


def chunk_paged(q, k_pages, v_pages, block_table, start, out=None, stream=None, check=False):
    """Chunked forward over a paged cache: q [B,Hq,L,128] at positions start..; pools
    [num_pages,Hkv,page_size,128]; block_table int32 [B,pages_per_seq] on the device."""
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _check(t, n)
    _check_i32(block_table, "block_table")
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, L, num_pages, page_size, pps = shapes.chunk_paged(
        q.shape, k_pages.shape, v_pages.shape, block_table.shape, int(start), None if out is None else out.shape)
    o = _out(q, out)
    _finish(kb_attn_chunk_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), o.data_ptr(), B, Hq, Hkv, L,
                                int(start), block_table.data_ptr(), pps, page_size, num_pages, _stream(stream)),
            "kb_attn_chunk_paged", check, stream)
    return o


def chunk_varlen(q, k, v, starts, lens, out=None, block_table=None, stream=None, check=False):
    """Ragged batch: q [B,Hq,L_max,128]; per-sequence starts/lens int32 [B] on the device; k/v either
    contiguous caches [B,Hkv,cap,128] or, with block_table [B,pages_per_seq], pools [num_pages,Hkv,page,128]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    for t, n in ((starts, "starts"), (lens, "lens")) + (((block_table, "block_table"),) if block_table is not None
                                                         else ()):
        _check_i32(t, n)
    if out is not None:
        _check(out, "out")
    sz = shapes.varlen(q.shape, k.shape, v.shape, starts.shape, lens.shape,
                       None if block_table is None else block_table.shape, None if out is None else out.shape)
    o = _out(q, out)
    if block_table is None:
        B, Hq, Hkv, L_max, cap = sz
        st = kb_attn_chunk_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, L_max,
                                  starts.data_ptr(), lens.data_ptr(), cap, None, 0, 0, 0, _stream(stream))
    else:
        B, Hq, Hkv, L_max, num_pages, page_size, pps = sz
        st = kb_attn_chunk_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, L_max,
                                  starts.data_ptr(), lens.data_ptr(), 0, block_table.data_ptr(), pps, page_size,
                                  num_pages, _stream(stream))
    _finish(st, "kb_attn_chunk_varlen", check, stream)
    return o


def check_device_status(stream=None):
    """Wait for `stream`, then raise KBError if a kernel since the last check gave up on a wait
    (KB_ERR_TIMEOUT) or found a device-resident argument out of range (KB_ERR_INVALID_ARG)."""
    _raise(kb_attn_check_device_status(_stream(stream)), "kb_attn_check_device_status")


def prefill_lse(q, k, v, out=None, lse=None, stream=None, check=False):
    """Training forward: (o, lse) with o bit-identical to prefill and lse [B,Hq,S] float32 the
    natural-log log-sum-exp of each row's scaled scores."""
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, S = shapes.prefill(q.shape, k.shape, v.shape, None if out is None else out.shape)
    o = _out(q, out)
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_f32(lse, "lse")
    shapes.vector_f32("lse", lse.shape, B, Hq, S)
    _finish(kb_attn_prefill_lse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv,
                                S, _stream(stream)), "kb_attn_prefill_lse", check, stream)
    return o, lse


def backward(q, k, v, o, dout, lse, delta=None, dq=None, dk=None, dv=None, stream=None, check=False):
    """Gradients (dq, dk, dv) of the whole-sequence causal prefill for output gradient dout; o and
    lse from prefill_lse.  Also returns delta [B,Hq,S] float32 = rowsum(dout * o)."""
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _check(t, n)
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        if t is not None:
            _check(t, n)
    B, Hq, Hkv, S = shapes.backward(q.shape, k.shape, v.shape, o.shape, dout.shape,
                                    None if dq is None else dq.shape, None if dk is None else dk.shape,
                                    None if dv is None else dv.shape)
    _check_f32(lse, "lse")
    shapes.vector_f32("lse", lse.shape, B, Hq, S)
    delta = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device) if delta is None else delta
    _check_f32(delta, "delta")
    shapes.vector_f32("delta", delta.shape, B, Hq, S)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _finish(kb_attn_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                             delta.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, S,
                             _stream(stream)), "kb_attn_backward", check, stream)
    return dq, dk, dv, delta


def _workspace(nbytes, device, workspace):
    torch = _torch()
    if workspace is None:
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    _on_current_device(workspace, "workspace")
    return workspace


def prefill_seg(q, k, v, seg_tiles, out=None, stream=None, check=False):
    """Segmented-mode prefill (segments of seg_tiles 128-key tiles, folded left to right)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, S = shapes.prefill(q.shape, k.shape, v.shape, None if out is None else out.shape)
    o = _out(q, out)
    _finish(kb_attn_prefill_seg(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, S,
                                int(seg_tiles), _stream(stream)), "kb_attn_prefill_seg", check, stream)
    return o


def chunk_seg(q, k, v, start, seg_tiles, out=None, workspace=None, stream=None, check=False):
    """Segmented-mode chunk: q [B,Hq,L,128] at positions start.., caches [B,Hkv,cap,128]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, L, cap = shapes.chunk(q.shape, k.shape, v.shape, int(start), None if out is None else out.shape)
    o = _out(q, out)
    ws = _workspace(kb_attn_seg_workspace_bytes(B, Hq, L, int(start), int(seg_tiles)), q.device, workspace)
    _finish(kb_attn_chunk_seg(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, L, int(start), cap,
                              int(seg_tiles), ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
            "kb_attn_chunk_seg", check, stream)
    return o


def decode_seg(q, k, v, ctx_len, seg_tiles, out=None, workspace=None, stream=None, check=False):
    """Segmented-mode decode: q [B,Hq,1,128] at position ctx_len-1."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, cap = shapes.decode(q.shape, k.shape, v.shape, int(ctx_len), None if out is None else out.shape)
    o = _out(q, out)
    ws = _workspace(kb_attn_seg_workspace_bytes(B, Hq, 1, int(ctx_len) - 1, int(seg_tiles)), q.device, workspace)
    _finish(kb_attn_decode_seg(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, int(ctx_len), cap,
                               int(seg_tiles), ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
            "kb_attn_decode_seg", check, stream)
    return o


def decode_seg_static(q, k, v, ctx_len, seg_tiles, out=None, stream=None, check=False):
    """Segmented-mode decode with the library's own scratch (no workspace argument, no allocation).
    Calls that overlap on the GPU share that scratch and must not run at the same time."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if out is not None:
        _check(out, "out")
    B, Hq, Hkv, cap = shapes.decode(q.shape, k.shape, v.shape, int(ctx_len), None if out is None else out.shape)
    o = _out(q, out)
    _finish(kb_attn_decode_seg_static(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv,
                                      int(ctx_len), cap, int(seg_tiles), _stream(stream)),
            "kb_attn_decode_seg_static", check, stream)
    return o


# ------------------------------------------------ rotation, cache append, block selection

def _check_view(t, name, device):
    """A [*, *, *, 128] view whose last dimension is contiguous: slices of a fused projection need no copy."""
    torch = _torch()
    try:
        if t.dtype is torch.bfloat16 and t.get_device() == device and not t.data_ptr() % 16:
            b, h, l, d = t.stride()
            if d == 1 and not (b | h | l) & 7:
                return
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dimensions [batch, heads, seq, head_dim]")
    if t.stride(3) != 1 or t.stride(0) % 8 or t.stride(1) % 8 or t.stride(2) % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name} must have a contiguous last dimension, strides that are multiples of 8 and 16-byte "
                         f"alignment, got strides {t.stride()}")
    _on_current_device(t, name)


# A one-token call runs for a few microseconds on the GPU, so what a call costs on the host counts: a tensor that
# passes the tests of _plain needs no closer look, shape rules are pure functions of shapes and remembered by them, and
# the current stream's handle is read without making a stream object.

def _plain(t, dtype, device):
    try:
        return t.dtype is dtype and t.get_device() == device and t.is_contiguous()
    except AttributeError:
        return False


def _need_bf16(t, name, device, ndim=4):
    if not _plain(t, _torch().bfloat16, device):
        _check(t, name, ndim)


def _need_i32(t, name, device):
    if t is not None and not _plain(t, _torch().int32, device):
        _check_i32(t, name)


def _need_f32(t, name, device):
    if t is not None and not _plain(t, _torch().float32, device):
        _check_f32(t, name)


_stride_array = functools.lru_cache(maxsize=1024)(lambda *strides: (ctypes.c_longlong * len(strides))(*strides))
_shapes_append = functools.lru_cache(maxsize=1024)(shapes.append)
_shapes_rope = functools.lru_cache(maxsize=1024)(shapes.rope)
_shapes_select = functools.lru_cache(maxsize=1024)(shapes.select)
_shapes_sparse = functools.lru_cache(maxsize=1024)(shapes.sparse)
_shapes_backward = functools.lru_cache(maxsize=1024)(shapes.backward)


def _stride3(t):
    return (0, 0, 0) if t is None else t.stride()[:3]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _shape(t):
    return None if t is None else t.shape


def _device():
    return _torch().cuda.current_device()


def _handle(stream, device):
    """The stream's handle; None: that of the current device's current stream."""
    return _torch()._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream`, from that stream's memory: the allocator may hand out memory that an earlier
    owner's kernels on another stream still use."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _per_sequence(B, t, name):
    if t is not None and t.shape != (B,):
        shapes.per_sequence(B, **{name: t.shape})


def rope_table(n_pos, rot_dim=128, theta=10000.0, inv_freq=None, device=None, stream=None):
    """Cosines and sines of position * inv_freq for positions 0..n_pos-1: float32 [n_pos, rot_dim/2, 2].  inv_freq
    (float64 [rot_dim/2]) defaults to theta ** (-2 i / rot_dim); angles are formed in 64 bits."""
    torch = _torch()
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if inv_freq is None:
        inv_freq = float(theta) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    if inv_freq.dim() != 1 or 2 * inv_freq.numel() != rot_dim:
        raise ValueError(f"inv_freq must have shape ({rot_dim // 2},), got {tuple(inv_freq.shape)}")
    with torch.cuda.stream(stream):
        inv_freq = inv_freq.to(device=device, dtype=torch.float64).contiguous()
        table = torch.empty((int(n_pos), rot_dim // 2, 2), dtype=torch.float32, device=device)
    shapes.rope_table(table.shape)
    _on_current_device(table, "table")
    _raise(kb_attn_rope_table(table.data_ptr(), int(n_pos), int(rot_dim), inv_freq.data_ptr(), _stream(stream)),
           "kb_attn_rope_table")
    return table


def rope(x, table, start=0, inverse=False, interleaved=False, out=None, stream=None, check=False):
    """Rotate x [B,H,L,128] (any strides, last dimension contiguous) by its positions start..start+L-1; inverse=True
    rotates by the negative angle, which turns the gradient of the result into the gradient of x."""
    device = _device()
    _check_view(x, "x", device)
    if not _plain(table, _torch().float32, device):
        _check_f32(table, "table")
    if out is not None:
        _need_bf16(out, "out", device)
    start = int(start)
    B, H, L, n_pos, rot_dim = _shapes_rope(x.shape, table.shape, start, _shape(out))
    o = _empty((B, H, L, 128), x.dtype, x.device, stream) if out is None else out
    _finish(kb_attn_rope(x.data_ptr(), _stride_array(*x.stride()[:3]), o.data_ptr(), table.data_ptr(), n_pos, rot_dim,
                         bool(interleaved), bool(inverse), B, H, L, start, _handle(stream, device)), "kb_attn_rope",
            check, stream)
    return o


def _append(q, k, v, k_cache, v_cache, table, start, starts, lens, block_table, boxes, interleaved, out, stream, check):
    device = _device()
    if q is not None:
        _check_view(q, "q", device)
    _check_view(k, "k", device)
    _check_view(v, "v", device)
    _need_bf16(k_cache, "k_cache", device)
    _need_bf16(v_cache, "v_cache", device)
    _need_f32(table, "table", device)
    _need_i32(starts, "starts", device)
    _need_i32(lens, "lens", device)
    _need_i32(block_table, "block_table", device)
    if boxes is not None:
        _need_bf16(boxes, "boxes", device, 5)
    if out is not None:
        _need_bf16(out, "out", device)
    B, Hq, Hkv, L, cap, num_pages, page, pps, n_pos, rot_dim = _shapes_append(
        _shape(q), k.shape, v.shape, k_cache.shape, v_cache.shape, _shape(table), _shape(boxes), _shape(block_table),
        _shape(out))
    _per_sequence(B, starts, "starts")
    _per_sequence(B, lens, "lens")
    if starts is None and not 0 <= start <= cap - L:
        raise ValueError(f"positions {start}..{start + L - 1} must lie in the cache's 0..{cap - 1}")
    if starts is None and table is not None and start > n_pos - L:
        raise ValueError(f"positions {start}..{start + L - 1} must lie in the table's 0..{n_pos - 1}")
    if q is not None and out is None:
        out = _empty((B, Hq, L, 128), q.dtype, q.device, stream)
    _finish(kb_attn_append(_ptr(q), k.data_ptr(), v.data_ptr(), _stride_array(*_stride3(q), *_stride3(k), *_stride3(v)),
                           _ptr(out), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(boxes), _ptr(table), n_pos, rot_dim,
                           bool(interleaved), B, Hq, Hkv, L, start, _ptr(starts), _ptr(lens), cap, _ptr(block_table),
                           pps, page, num_pages, _handle(stream, device)), "kb_attn_append", check, stream)
    return out


def append(q, k, v, k_cache, v_cache, table, start, boxes=None, interleaved=False, out=None, stream=None, check=False):
    """Append k, v [B,Hkv,L,128] to caches [B,Hkv,cap,128] at positions start..start+L-1, k and q [B,Hq,L,128]
    rotated by them (table from rope_table, None: not rotated), and widen the boxes of the touched key blocks.
    Returns the rotated q, contiguous (None without q).  q, k, v may be slices of one fused projection."""
    return _append(q, k, v, k_cache, v_cache, table, int(start), None, None, None, boxes, interleaved, out, stream,
                   check)


def append_varlen(q, k, v, k_cache, v_cache, table, starts, lens=None, block_table=None, boxes=None, interleaved=False,
                  out=None, stream=None, check=False):
    """append with a start (and row count, default all rows) per sequence, int32 [B] on the device; with block_table
    [B,pages_per_seq] the caches are pools [num_pages,Hkv,page_size,128].  Rows of the result from lens[b] on are left
    as they were."""
    if starts is None:
        raise TypeError("starts must be a contiguous int32 CUDA tensor")
    return _append(q, k, v, k_cache, v_cache, table, 0, starts, lens, block_table, boxes, interleaved, out, stream,
                   check)


def block_boxes(k, kv_len=None, kv_lens=None, block_table=None, boxes=None, stream=None, check=False):
    """Boxes (upper and lower bound per channel) of the blocks of 128 keys of a cache [B,Hkv,cap,128], or of pools with
    block_table: of its first kv_len keys (default: all), or kv_lens[b] of sequence b.  Returns bf16
    [B or num_pages, Hkv, blocks, 2, 128]; blocks beyond are zero in a new tensor and left as they were in `boxes`."""
    torch = _torch()
    device = _device()
    _need_bf16(k, "k", device)
    _need_i32(kv_lens, "kv_lens", device)
    _need_i32(block_table, "block_table", device)
    if boxes is not None:
        _need_bf16(boxes, "boxes", device, 5)
    B, Hkv, cap, num_pages, page, pps, box = shapes.block_boxes(k.shape, _shape(block_table), _shape(boxes))
    _per_sequence(B, kv_lens, "kv_lens")
    kv_len = cap if kv_len is None else int(kv_len)
    if not 1 <= kv_len <= cap:
        raise ValueError(f"kv_len must lie in 1..{cap} (the cache capacity), got {kv_len}")
    if boxes is None:
        boxes = _empty(box, torch.bfloat16, k.device, stream)
        with torch.cuda.stream(stream):
            boxes.zero_()
    _finish(kb_attn_block_boxes(k.data_ptr(), boxes.data_ptr(), B, Hkv, kv_len, _ptr(kv_lens), cap, _ptr(block_table),
                                pps, page, num_pages, _handle(stream, device)), "kb_attn_block_boxes", check, stream)
    return boxes


def _select(q, boxes, start, starts, lens, n, keep_first, keep_last, block_table, out, stream, check):
    torch = _torch()
    device = _device()
    _need_bf16(q, "q", device)
    _need_bf16(boxes, "boxes", device, 5)
    _need_i32(starts, "starts", device)
    _need_i32(lens, "lens", device)
    _need_i32(block_table, "block_table", device)
    _need_i32(out, "out", device)
    B, Hq, Hkv, L, per_plane, num_pages, page, pps = _shapes_select(q.shape, boxes.shape, n, keep_first, keep_last,
                                                                    _shape(block_table), _shape(out))
    _per_sequence(B, starts, "starts")
    _per_sequence(B, lens, "lens")
    if starts is None and not 0 <= start <= per_plane * shapes.BLOCK - L:
        raise ValueError(f"positions {start}..{start + L - 1} must lie in the boxes' 0..{per_plane * shapes.BLOCK - 1}")
    if out is None:
        out = _empty((B, Hkv, L, n), torch.int32, q.device, stream)
    _finish(kb_attn_select_blocks(q.data_ptr(), boxes.data_ptr(), out.data_ptr(), B, Hq, Hkv, L, n, keep_first,
                                  keep_last, start, _ptr(starts), _ptr(lens), per_plane, _ptr(block_table), pps, page,
                                  num_pages, _handle(stream, device)), "kb_attn_select_blocks", check, stream)
    return out


def select_blocks(q, boxes, start, n, keep_first=1, keep_last=1, out=None, stream=None, check=False):
    """The n key blocks each row of q [B,Hq,L,128] (positions start..) attends to, by the boxes [B,Hkv,blocks,2,128]
    of the keys: int32 [B,Hkv,L,n], ascending, -1 behind the last.  The first keep_first and last keep_last of a row's
    blocks are always taken."""
    return _select(q, boxes, int(start), None, None, int(n), int(keep_first), int(keep_last), None, out, stream, check)


def select_blocks_varlen(q, boxes, starts, n, lens=None, block_table=None, keep_first=1, keep_last=1, out=None,
                         stream=None, check=False):
    """select_blocks with a start (and row count) per sequence, int32 [B] on the device, and optionally the boxes of
    paged pools [num_pages,Hkv,page_size/128,2,128] with block_table [B,pages_per_seq].  Rows from lens[b] on are left
    as they were."""
    if starts is None:
        raise TypeError("starts must be a contiguous int32 CUDA tensor")
    return _select(q, boxes, 0, starts, lens, int(n), int(keep_first), int(keep_last), block_table, out, stream, check)


# ------------------------------------------------------------- block-sparse attention

def _sparse_args(device, q, k, v, blocks, block_table=None, out=None, positions=()):
    _need_bf16(q, "q", device)
    _need_bf16(k, "k", device)
    _need_bf16(v, "v", device)
    if not _plain(blocks, _torch().int32, device):
        _check_i32(blocks, "blocks")
    _need_i32(block_table, "block_table", device)
    if out is not None:
        _need_bf16(out, "out", device)
    sz = _shapes_sparse(q.shape, k.shape, v.shape, blocks.shape, _shape(block_table), _shape(out))
    for t, name in positions:
        _need_i32(t, name, device)
        _per_sequence(sz[0], t, name)
    return sz


def _stream_workspace(nbytes, device, workspace, stream):
    if workspace is not None:
        return _workspace(nbytes, device, workspace)
    return _empty(max(int(nbytes), 256), _torch().uint8, device, stream)


def _sparse_workspace(B, Hkv, L, n, cap, device, workspace, stream):
    return _stream_workspace(kb_attn_sparse_workspace_bytes(B, Hkv, L, n, cap), device, workspace, stream)


def _sparse_chunk(q, k, v, start, starts, lens, blocks, block_table, out, workspace, stream, check):
    device = _device()
    B, Hq, Hkv, L, n, cap, num_pages, page, pps = _sparse_args(device, q, k, v, blocks, block_table, out,
                                                               ((starts, "starts"), (lens, "lens")))
    if starts is None and not 0 <= start <= cap - L:
        raise ValueError(f"positions {start}..{start + L - 1} must lie in the cache's 0..{cap - 1}")
    o = _empty(q.shape, q.dtype, q.device, stream) if out is None else out
    ws = _sparse_workspace(B, Hkv, L, n, cap, q.device, workspace, stream)
    _finish(kb_attn_sparse_chunk(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), blocks.data_ptr(), n, B, Hq,
                                 Hkv, L, start, _ptr(starts), _ptr(lens), cap, _ptr(block_table), pps, page, num_pages,
                                 ws.data_ptr(), ws.numel() * ws.element_size(), _handle(stream, device)),
            "kb_attn_sparse_chunk", check, stream)
    return o


def sparse_chunk(q, k, v, start, blocks, out=None, workspace=None, stream=None, check=False):
    """chunk over listed key blocks: row i of q [B,Hq,L,128] (position start + i) sees the keys of blocks
    blocks[b, g, i] (int32 [B,Hkv,L,n], -1 for none) up to its position.  k/v caches [B,Hkv,cap,128]."""
    return _sparse_chunk(q, k, v, int(start), None, None, blocks, None, out, workspace, stream, check)


def sparse_chunk_varlen(q, k, v, starts, blocks, lens=None, block_table=None, out=None, workspace=None, stream=None,
                        check=False):
    """sparse_chunk with a start (and row count) per sequence, int32 [B] on the device, and optionally paged pools with
    block_table [B,pages_per_seq].  Rows from lens[b] on are left as they were."""
    if starts is None:
        raise TypeError("starts must be a contiguous int32 CUDA tensor")
    return _sparse_chunk(q, k, v, 0, starts, lens, blocks, block_table, out, workspace, stream, check)


def _sparse_decode(q, k, v, ctx_len, ctx_lens, blocks, block_table, out, stream, check):
    device = _device()
    B, Hq, Hkv, L, n, cap, num_pages, page, pps = _sparse_args(device, q, k, v, blocks, block_table, out,
                                                               ((ctx_lens, "ctx_lens"),))
    if L != 1:
        raise ValueError(f"decode takes one query row per (batch, head), got {L}")
    if ctx_lens is None and not 1 <= ctx_len <= cap:
        raise ValueError(f"ctx_len must lie in 1..{cap} (the cache capacity), got {ctx_len}")
    o = _empty(q.shape, q.dtype, q.device, stream) if out is None else out
    _finish(kb_attn_sparse_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), blocks.data_ptr(), n, B, Hq,
                                  Hkv, ctx_len, _ptr(ctx_lens), cap, _ptr(block_table), pps, page, num_pages,
                                  _handle(stream, device)), "kb_attn_sparse_decode", check, stream)
    return o


def sparse_decode(q, k, v, ctx_len, blocks, out=None, stream=None, check=False):
    """decode over listed key blocks: q [B,Hq,1,128] at position ctx_len-1, blocks int32 [B,Hkv,1,n]."""
    return _sparse_decode(q, k, v, int(ctx_len), None, blocks, None, out, stream, check)


def sparse_decode_paged(q, k_pages, v_pages, block_table, ctx_lens, blocks, out=None, stream=None, check=False):
    """decode_paged over listed key blocks: blocks int32 [B,Hkv,1,n], indices within each sequence."""
    for t, n in ((block_table, "block_table"), (ctx_lens, "ctx_lens")):
        _check_i32(t, n)
    return _sparse_decode(q, k_pages, v_pages, 0, ctx_lens, blocks, block_table, out, stream, check)


def sparse_prefill_lse(q, k, v, blocks, out=None, lse=None, workspace=None, stream=None, check=False):
    """Training forward over listed key blocks of a whole sequence: (o, lse) as prefill_lse; a row that lists nothing
    has o = 0 and lse = -inf."""
    torch = _torch()
    device = _device()
    B, Hq, Hkv, S, n, cap, _, _, _ = _sparse_args(device, q, k, v, blocks, None, out)
    shapes.prefill(q.shape, k.shape, v.shape)
    o = _empty(q.shape, q.dtype, q.device, stream) if out is None else out
    lse = _empty((B, Hq, S), torch.float32, q.device, stream) if lse is None else lse
    _check_f32(lse, "lse")
    shapes.vector_f32("lse", lse.shape, B, Hq, S)
    ws = _sparse_workspace(B, Hkv, S, n, cap, q.device, workspace, stream)
    _finish(kb_attn_sparse_prefill_lse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                       blocks.data_ptr(), n, B, Hq, Hkv, S, ws.data_ptr(),
                                       ws.numel() * ws.element_size(), _handle(stream, device)),
            "kb_attn_sparse_prefill_lse", check, stream)
    return o, lse


def sparse_backward(q, k, v, o, dout, lse, blocks, delta=None, dq=None, dk=None, dv=None, workspace=None, stream=None,
                    check=False):
    """Gradients (dq, dk, dv) of sparse_prefill_lse for output gradient dout; o, lse from it, blocks as given to it.
    Also returns delta [B,Hq,S] float32 = rowsum(dout * o)."""
    torch = _torch()
    device = _device()
    B, Hq, Hkv, S, n, _, _, _, _ = _sparse_args(device, q, k, v, blocks)
    for t, name in ((o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        if t is not None or name in ("o", "dout"):
            _need_bf16(t, name, device)
    _shapes_backward(q.shape, k.shape, v.shape, o.shape, dout.shape, _shape(dq), _shape(dk), _shape(dv))
    delta = _empty((B, Hq, S), torch.float32, q.device, stream) if delta is None else delta
    for t, name in ((lse, "lse"), (delta, "delta")):
        _check_f32(t, name)
        shapes.vector_f32(name, t.shape, B, Hq, S)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(k.shape, k.dtype, k.device, stream) if dk is None else dk
    dv = _empty(v.shape, v.dtype, v.device, stream) if dv is None else dv
    ws = _stream_workspace(kb_attn_sparse_backward_workspace_bytes(B, Hkv, S, n), q.device, workspace, stream)
    _finish(kb_attn_sparse_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                                    lse.data_ptr(), delta.data_ptr(), blocks.data_ptr(), n, dq.data_ptr(),
                                    dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, S, ws.data_ptr(),
                                    ws.numel() * ws.element_size(), _handle(stream, device)),
            "kb_attn_sparse_backward", check, stream)
    return dq, dk, dv, delta
