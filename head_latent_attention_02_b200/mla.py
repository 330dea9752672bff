"""Python binding of libmla (include/mla.h): argument marshalling only.

Every step runs in the library's CUDA kernels; this module turns torch
tensors into pointers and sizes, calls the C ABI and raises on a non-OK
status.  It fails loudly when libmla.so is missing -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "mla.h")

MLA_F32, MLA_BF16 = 0, 1
STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_BAD_INDEX"}


class MLAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32),
                ("d_n", ctypes.c_int32), ("d_v", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("rope_base", ctypes.c_double)]


_lib = None
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_pi32 = ctypes.POINTER(_i32)
_SIGS = {
    "mla_abi_version": ([], _i32),
    "mla_status_str": ([_i32], ctypes.c_char_p),
    "mla_get_status": ([_vp], _i32),
    "mla_absorb_q": ([ctypes.POINTER(Dims), _i32, _vp, _vp, _vp, ctypes.POINTER(_i32), _i32, _vp,
                      _vp, _vp], _i32),
    "mla_decode": ([ctypes.POINTER(Dims), _i32, _i32, _vp, _i32, _vp, _i32, _vp, _i64, _vp, _i32,
                    _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "mla_decode_workspace_size": ([ctypes.POINTER(Dims), _i32, _i32, _i32, _i32], _sz),
    "mla_decode_static_ws": ([ctypes.POINTER(Dims), _i32, _i32, _vp, _i32, _vp, _i32, _vp, _i64,
                              _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp], _i32),
    "mla_decode_static_ws_init": ([], _i32),
    "mla_merge_lse": ([_i32, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "mla_out_proj": ([ctypes.POINTER(Dims), _i32, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "mla_append_rows": ([ctypes.POINTER(Dims), _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i64,
                         _vp, _i32, _vp, ctypes.c_float, _vp, _vp], _i32),
    "mla_qknorm_query": ([ctypes.POINTER(Dims), _i32, _vp, _vp, _vp, ctypes.c_float, _vp, _vp],
                         _i32),
    "mla_qknorm_key_gram": ([ctypes.POINTER(Dims), _vp, _vp, _vp], _i32),
    "mla_debug_wait_probe": ([_i64, _vp, _vp], _i32),
    "mla_pack_rows": ([ctypes.POINTER(Dims), _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp], _i32),
    "mla_decode_lowbit": ([ctypes.POINTER(Dims), _i32, _i32, _i32, _i32, _vp, _i32, _vp, _i32,
                           _vp, _vp, _vp, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp,
                           _vp, _vp], _i32),
    "mla_lowbit_dequant_bytes": ([ctypes.POINTER(Dims), _i64], _sz),
    "mla_dequant_rows": ([ctypes.POINTER(Dims), _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp], _i32),
    "mla_decode_lowbit_tc": ([ctypes.POINTER(Dims), _i32, _i32, _i32, _i32, _vp, _i32, _vp, _i32,
                              _vp, _vp, _vp, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp,
                              _vp, _vp, _sz, _vp, _sz, _vp], _i32),
    "mla_decode_qknorm": ([ctypes.POINTER(Dims), _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64,
                           _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "mla_rope_axes": ([ctypes.POINTER(Dims), _i32, _i32, _vp, _i64, _i64, _vp, _i32, _pi32, _i32,
                       _vp, _i64, _i64, _vp], _i32),
    "mla_append_tokens": ([ctypes.POINTER(Dims), _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i32, _pi32,
                           _vp, ctypes.c_float, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _i32, _vp],
                          _i32),
    "mla_chunk_attn": ([ctypes.POINTER(Dims), _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp,
                        _i32, _vp, _i32, _pi32, _i32, _i64, _vp, _vp, _vp, _sz, _vp], _i32),
    "mla_chunk_workspace_size": ([ctypes.POINTER(Dims), _i32, _i32, _i32, _i32, _i32, _i64], _sz),
    "mla_linear": ([_i32, _i32, _i32, _i32, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _i64,
                    _vp, _sz, _vp], _i32),
    "mla_linear_workspace_size": ([_i32, _i32, _i32, _i32], _sz),
}


def lib() -> ctypes.CDLL:
    """Load libmla.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmla.so not built at {LIB_PATH}: run "
                               "`python -m head_latent_attention_02_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def header_symbols() -> list:
    """Entry points declared in include/mla.h."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\*]+\s+\*?(mla_\w+)\s*\(", txt, re.M)))


def make_dims(wl, dtype: Optional[int] = None) -> Dims:
    return Dims(wl.H, wl.d_c, wl.d_r, wl.d_n, wl.d_v, wl.d_model, 64,
                (MLA_BF16 if wl.dtype == "bf16" else MLA_F32) if dtype is None else dtype,
                wl.scale, wl.rope_base)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _s(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, code: int):
    if code != 0:
        raise MLAError(fn, code)


def status_str(code: int) -> str:
    return lib().mla_status_str(code).decode()


def get_status(stream=None) -> int:
    """Waits for the stream and returns (and clears) the device status word."""
    return int(lib().mla_get_status(_s(stream)))


def absorb_q(dims: Dims, q_nope, q_rope, q_pos, deltas: Sequence[int], w_uk, q_abs, stream=None):
    n_q = q_nope.shape[0]
    arr = (_i32 * len(deltas))(*[int(d) for d in deltas])
    _check("mla_absorb_q", lib().mla_absorb_q(ctypes.byref(dims), n_q, _p(q_nope), _p(q_rope),
                                              _p(q_pos), arr, len(deltas), _p(w_uk), _p(q_abs),
                                              _s(stream)))


def workspace_size(dims: Dims, B: int, s_q: int, n_h: int, n_ver: int = 1) -> int:
    return int(lib().mla_decode_workspace_size(ctypes.byref(dims), B, s_q, n_ver, n_h))


def decode(dims: Dims, B: int, s_q: int, q_abs, n_ver: int, head_ids, n_h: int, cache,
           block_table, segs, q_pos, o_lat, lse, workspace, gather_rows=None, n_gather=None,
           stream=None):
    """mla_decode; ``head_ids`` is an int32 device tensor of n_h head ids, or
    None for heads 0 .. n_h-1."""
    n_pages = cache.shape[0]
    max_pages = block_table.shape[1]
    max_segs = segs.shape[1]
    max_gather = gather_rows.shape[1] if gather_rows is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("mla_decode", lib().mla_decode(
        ctypes.byref(dims), B, s_q, _p(q_abs), n_ver, _p(head_ids), n_h, _p(cache), n_pages,
        _p(block_table), max_pages, _p(segs), max_segs, _p(gather_rows), _p(n_gather),
        max_gather, _p(q_pos), _p(o_lat), _p(lse), _p(workspace), ws_bytes, _s(stream)))


def decode_static_ws(dims: Dims, B: int, s_q: int, q_abs, n_ver: int, head_ids, n_h: int, cache,
                     block_table, segs, q_pos, o_lat, lse, gather_rows=None, n_gather=None,
                     stream=None):
    """mla_decode with the library's fixed scratch array instead of a workspace."""
    max_gather = gather_rows.shape[1] if gather_rows is not None else 0
    _check("mla_decode_static_ws", lib().mla_decode_static_ws(
        ctypes.byref(dims), B, s_q, _p(q_abs), n_ver, _p(head_ids), n_h, _p(cache), cache.shape[0],
        _p(block_table), block_table.shape[1], _p(segs), segs.shape[1], _p(gather_rows),
        _p(n_gather), max_gather, _p(q_pos), _p(o_lat), _p(lse), _s(stream)))


def decode_static_ws_init():
    """Loads the static scratch array on the current device."""
    _check("mla_decode_static_ws_init", lib().mla_decode_static_ws_init())


def merge_lse(n_q: int, H: int, head_ids, n_h: int, d: int, o_a, lse_a, o_b, lse_b, o, lse,
              stream=None):
    _check("mla_merge_lse", lib().mla_merge_lse(n_q, H, _p(head_ids), n_h, d, _p(o_a), _p(lse_a),
                                                _p(o_b), _p(lse_b), _p(o), _p(lse), _s(stream)))


def out_proj(dims: Dims, o_lat, w_uv, w_o, v, out, stream=None):
    n_q = o_lat.shape[0]
    _check("mla_out_proj", lib().mla_out_proj(ctypes.byref(dims), n_q, _p(o_lat), _p(w_uv),
                                              _p(w_o), _p(v), _p(out), _s(stream)))


def append_rows(dims, c_new, k_rope_raw, cache_pos, seq, row, cache, block_table,
                key_gram=None, qk_eps=0.0, key_inv_rms=None, stream=None):
    """mla_append_rows: entries i -> cache row (seq[i], row[i]) = [c | R(cache_pos) k_raw]
    (QK-normed caches: with key_gram, also key_inv_rms and a rescaled k_rope)."""
    _check("mla_append_rows", lib().mla_append_rows(
        ctypes.byref(dims), c_new.shape[0], _p(c_new), _p(k_rope_raw), _p(cache_pos), _p(seq),
        _p(row), block_table.shape[0], _p(cache), cache.shape[0], _p(block_table),
        block_table.shape[1], _p(key_gram), qk_eps, _p(key_inv_rms), _s(stream)))


def qknorm_query(dims, q_nope, g_q, g_k, eps, q_out, stream=None):
    _check("mla_qknorm_query", lib().mla_qknorm_query(
        ctypes.byref(dims), q_nope.shape[0], _p(q_nope), _p(g_q), _p(g_k), eps, _p(q_out),
        _s(stream)))


def qknorm_key_gram(dims, w_uk, gram, stream=None):
    _check("mla_qknorm_key_gram", lib().mla_qknorm_key_gram(ctypes.byref(dims), _p(w_uk),
                                                            _p(gram), _s(stream)))


def decode_qknorm(dims, B, s_q, q_abs, n_ver, head_ids, n_h, cache, key_inv_rms, block_table,
                  segs, q_pos, o_lat, lse, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("mla_decode_qknorm", lib().mla_decode_qknorm(
        ctypes.byref(dims), B, s_q, _p(q_abs), n_ver, _p(head_ids), n_h, _p(cache),
        _p(key_inv_rms), cache.shape[0], _p(block_table), block_table.shape[1], _p(segs),
        segs.shape[1], _p(q_pos), _p(o_lat), _p(lse), _p(workspace), ws_bytes, _s(stream)))


def pack_rows(dims, bits_c, bits_r, rows, scale_c, scale_r, packed, stream=None):
    """mla_pack_rows: rows [n, d_c + d_r] -> packed codes [n, row bytes]."""
    _check("mla_pack_rows", lib().mla_pack_rows(ctypes.byref(dims), bits_c, bits_r,
                                                rows.shape[0], _p(rows), _p(scale_c),
                                                _p(scale_r), _p(packed), _s(stream)))


def decode_lowbit(dims, bits_c, bits_r, B, s_q, q_abs, n_ver, head_ids, n_h, cache, scale_c,
                  scale_r, block_table, segs, q_pos, o_lat, lse, gather_rows=None, n_gather=None,
                  stream=None):
    """mla_decode_lowbit over a packed pool cache [n_pages, 64, row bytes] (uint8)."""
    max_gather = gather_rows.shape[1] if gather_rows is not None else 0
    _check("mla_decode_lowbit", lib().mla_decode_lowbit(
        ctypes.byref(dims), bits_c, bits_r, B, s_q, _p(q_abs), n_ver, _p(head_ids), n_h,
        _p(cache), _p(scale_c), _p(scale_r), cache.shape[0], _p(block_table),
        block_table.shape[1], _p(segs), segs.shape[1], _p(gather_rows), _p(n_gather),
        max_gather, _p(q_pos), _p(o_lat), _p(lse), _s(stream)))


def lowbit_dequant_bytes(dims, n_pages):
    """mla_lowbit_dequant_bytes: bytes of a dequantised pool of n_pages pages."""
    return lib().mla_lowbit_dequant_bytes(ctypes.byref(dims), n_pages)


def dequant_rows(dims, bits_c, bits_r, packed, scale_c, scale_r, out, stream=None):
    """mla_dequant_rows: packed codes [n, row bytes] -> out [n, d_c + d_r] (dtype)."""
    _check("mla_dequant_rows", lib().mla_dequant_rows(ctypes.byref(dims), bits_c, bits_r,
                                                      packed.shape[0], _p(packed), _p(scale_c),
                                                      _p(scale_r), _p(out), _s(stream)))


def decode_lowbit_tc(dims, bits_c, bits_r, B, s_q, q_abs, n_ver, head_ids, n_h, cache, scale_c,
                     scale_r, block_table, segs, q_pos, o_lat, lse, dequant, workspace,
                     gather_rows=None, n_gather=None, stream=None):
    """mla_decode_lowbit_tc over a packed pool cache [n_pages, 64, row bytes]
    (uint8), dequantising into ``dequant`` and decoding with ``workspace``."""
    max_gather = gather_rows.shape[1] if gather_rows is not None else 0
    dq_bytes = dequant.numel() * dequant.element_size()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("mla_decode_lowbit_tc", lib().mla_decode_lowbit_tc(
        ctypes.byref(dims), bits_c, bits_r, B, s_q, _p(q_abs), n_ver, _p(head_ids), n_h,
        _p(cache), _p(scale_c), _p(scale_r), cache.shape[0], _p(block_table),
        block_table.shape[1], _p(segs), segs.shape[1], _p(gather_rows), _p(n_gather),
        max_gather, _p(q_pos), _p(o_lat), _p(lse), _p(dequant), dq_bytes, _p(workspace),
        ws_bytes, _s(stream)))


# ------------------------------------------------------------------ prompt chunks
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_TORCH_DTYPE = {MLA_F32: torch.float32, MLA_BF16: torch.bfloat16}


def _ints(values: Sequence[int]):
    return (_i32 * len(values))(*[int(v) for v in values])


def _bytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _want(t: Optional[torch.Tensor], name: str, dtype, shape=None):
    """Raises unless t (None passes) has the dtype and the sizes of ``shape`` (None: any)."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and (t.dim() != len(shape) or
                              any(w is not None and w != n for w, n in zip(shape, t.shape))):
        raise ValueError(f"{name} must have sizes {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t: Optional[torch.Tensor], name: str) -> int:
    """Stride between the rows of a matrix whose last axis is contiguous."""
    if t is None:
        return 0
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return max(t.stride(0), t.shape[1]) if t.shape[0] <= 1 else t.stride(0)


def rope_axes(dims: Dims, x, pos, sections: Sequence[int], out, inverse: bool = False, stream=None):
    """mla_rope_axes: x, out [n_tok, n_heads, d_r] views (any token and head strides), pos
    [len(sections), n_tok] int32; ``out`` may be ``x``."""
    n_tok, n_heads, d_r = x.shape
    dt = _TORCH_DTYPE.get(dims.dtype)
    _want(x, "x", dt, (None, None, dims.d_r))
    _want(out, "out", dt, (n_tok, n_heads, d_r))
    _want(pos, "pos", torch.int32, (len(sections), n_tok))
    if x.stride(2) != 1 or out.stride(2) != 1:
        raise ValueError("the last axis of x and out must be contiguous")
    _check("mla_rope_axes", lib().mla_rope_axes(
        ctypes.byref(dims), n_tok, n_heads, x.data_ptr(), x.stride(0), x.stride(1), _p(pos),
        len(sections), _ints(sections), int(inverse), out.data_ptr(), out.stride(0), out.stride(1),
        _s(stream)))


def append_tokens(dims: Dims, kv, tok_start, row0, pos, sections: Sequence[int], cache, block_table,
                  norm_weight=None, norm_eps: float = 0.0, bits: Optional[Sequence[int]] = None,
                  scale_c=None, scale_r=None, stream=None):
    """mla_append_tokens: kv [n_tok, d_c + d_r] rows (any row stride) into the pages of sequences
    tok_start describes; ``bits`` (bits_c, bits_r) for a packed pool, else rows of the dtype."""
    n_tok, B = kv.shape[0], row0.shape[0]
    _want(kv, "kv", _TORCH_DTYPE.get(dims.dtype), (None, dims.d_c + dims.d_r))
    _want(tok_start, "tok_start", torch.int32, (B + 1,))
    _want(row0, "row0", torch.int32, (B,))
    _want(pos, "pos", torch.int32, (len(sections), n_tok))
    _want(block_table, "block_table", torch.int32, (B, None))
    _want(norm_weight, "norm_weight", torch.float32, (dims.d_c,))
    _want(scale_c, "scale_c", torch.float32, (dims.d_c,))
    _want(scale_r, "scale_r", torch.float32, (dims.d_r,))
    bits_c, bits_r = bits if bits else (0, 0)
    if bits:
        _want(cache, "cache", torch.uint8, (None, 64, (dims.d_c * bits_c + dims.d_r * bits_r) // 8))
    else:
        _want(cache, "cache", _TORCH_DTYPE.get(dims.dtype), (None, 64, dims.d_c + dims.d_r))
    _check("mla_append_tokens", lib().mla_append_tokens(
        ctypes.byref(dims), B, n_tok, kv.data_ptr(), _rows(kv, "kv"), _p(tok_start), _p(row0),
        _p(pos), len(sections), _ints(sections), _p(norm_weight), norm_eps, bits_c, bits_r,
        _p(scale_c), _p(scale_r), _p(cache), cache.shape[0], _p(block_table), block_table.shape[1],
        _s(stream)))


def chunk_workspace_size(dims: Dims, B: int, n_tok: int, n_ver: int, max_pages: int, max_segs: int,
                         max_rows: int) -> int:
    return int(lib().mla_chunk_workspace_size(ctypes.byref(dims), B, n_tok, n_ver, max_pages,
                                              max_segs, max_rows))


def chunk_attn(dims: Dims, q, tok_start, q_pos, w_uk, w_uv, cache, block_table, segs,
               deltas: Sequence[int], max_rows: int, v, workspace, lse=None, stream=None):
    """mla_chunk_attn: q [n_tok, H, d_n + d_r] (rotary part rotated) over the cached rows of the
    sequences tok_start describes -> v [n_tok, H, d_v]; lse [n_tok, H] or None."""
    n_tok, B = q.shape[0], tok_start.shape[0] - 1
    dt = _TORCH_DTYPE.get(dims.dtype)
    _want(q, "q", dt, (None, dims.H, dims.d_n + dims.d_r))
    _want(tok_start, "tok_start", torch.int32, (B + 1,))
    _want(q_pos, "q_pos", torch.int32, (n_tok,))
    _want(w_uk, "w_uk", dt, (dims.H, dims.d_n, dims.d_c))
    _want(w_uv, "w_uv", dt, (dims.H, dims.d_v, dims.d_c))
    _want(cache, "cache", dt, (None, 64, dims.d_c + dims.d_r))
    _want(block_table, "block_table", torch.int32, (B, None))
    _want(segs, "segs", torch.int32, (B, None, 4))
    _want(v, "v", dt, (n_tok, dims.H, dims.d_v))
    _want(lse, "lse", torch.float32, (n_tok, dims.H))
    _check("mla_chunk_attn", lib().mla_chunk_attn(
        ctypes.byref(dims), B, n_tok, _p(q), _p(tok_start), _p(q_pos), _p(w_uk), _p(w_uv), _p(cache),
        cache.shape[0], _p(block_table), block_table.shape[1], _p(segs), segs.shape[1],
        _ints(deltas), len(deltas), max_rows, _p(v), _p(lse), _p(workspace), _bytes(workspace),
        _s(stream)))


def linear_workspace_size(x, w) -> int:
    """Bytes of workspace for linear(x, w, ...)."""
    dt = MLA_BF16 if x.dtype == torch.bfloat16 else MLA_F32
    return int(lib().mla_linear_workspace_size(dt, x.shape[0], w.shape[0], x.shape[1]))


def linear(x, w, out, bias=None, act: str = "none", residual=None, workspace=None, stream=None):
    """mla_linear: out [M, N] = act(x [M, K] w [N, K]^T + bias [N]) + residual [M, N]; matrices may
    have any row stride; ``out`` may be ``residual``."""
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be matrices")
    (M, K), N = x.shape, w.shape[0]
    _want(w, "w", x.dtype, (N, K))
    _want(out, "out", x.dtype, (M, N))
    _want(bias, "bias", torch.float32, (N,))
    _want(residual, "residual", x.dtype, (M, N))
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    _check("mla_linear", lib().mla_linear(
        MLA_BF16 if x.dtype == torch.bfloat16 else MLA_F32, M, N, K, x.data_ptr(), _rows(x, "x"),
        w.data_ptr(), _rows(w, "w"), _p(bias), ACTIVATIONS[act],
        None if residual is None else residual.data_ptr(), _rows(residual, "residual"),
        out.data_ptr(), _rows(out, "out"), _p(workspace), _bytes(workspace), _s(stream)))
