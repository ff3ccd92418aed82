"""Attention around a paged key-value cache: the binding of the ``qgemm_qk_rope_append``,
``qgemm_attn_decode`` and ``qgemm_attn_prefill`` entry points of ``include/qgemm.h``.

As in the rest of the package: argument marshalling only, on the current HIP stream of the tensors'
device, and no fallback. Shapes, types and devices are checked here; strides, alignment, ranges and
overlaps by the library, which raises ``QgemmError``.
"""

from __future__ import annotations

import ctypes
import functools
import math
import struct

from . import DT_BF16, DT_F16, DT_FP8, Workspace, _check, _default_ws, _torch, lib

__all__ = ["KVCache", "rope_table", "qk_rope_append", "attn_decode", "attn_prefill", "set_attn_splits",
           "attn_decode_workspace_bytes", "attn_prefill_workspace_bytes"]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]

# The argument structs of the *_call entry points, packed into bytes: one argument through ctypes costs about as much
# as all of a struct's fields.
_attn_call = struct.Struct("@P2q2PqPP4qqP2qPNP3if").pack
_append_call = struct.Struct("@P2qP2qP2q3Pq3P3qPP2qP4if4x").pack


@functools.lru_cache(maxsize=None)
def _dtypes():
    torch = _torch()
    return {torch.float16: DT_F16, torch.bfloat16: DT_BF16, torch.float8_e4m3fn: DT_FP8}


class KVCache:
    """A paged key-value cache: k and v are [pages][page_size][kv_heads][head_dim] tensors (or views with the last
    dimension contiguous, the same strides for both), float16, bfloat16 or float8_e4m3fn; an e4m3 code stands for its
    value times k_scale (keys) or v_scale (values). Holds references, copies nothing, and is fixed: the calls take its
    addresses, strides and scales as they were given here, so other ones need another KVCache (5 us)."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [pages][page_size][kv_heads][head_dim] of one type, device and strides")
        if k.dtype not in _dtypes():
            raise ValueError("the cache must be float16, bfloat16 or float8_e4m3fn")
        if not k.is_cuda:
            raise ValueError("tensor must live on the GPU")
        if k.stride(3) != 1:
            raise ValueError("a head's values must be contiguous")
        self.k, self.v, self.device = k, v, k.device
        self._index = k.get_device()   # the calls use this device's current stream
        # what every call looks up, at hand: calls are bound by their host time when they move little
        torch = _torch()
        self._int32_type, self._float32_type = torch.int32, torch.float32
        self._empty_like, self._stream = torch.empty_like, torch._C._cuda_getCurrentRawStream
        self._acts = {torch.float16: DT_F16, torch.bfloat16: DT_BF16}
        self._norm_shape = torch.Size((k.shape[3],))
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), self.num_pages, k.stride(0), k.stride(1), k.stride(2),
                                    self.page_size, self.kv_heads, self.head_dim, _dtypes()[k.dtype], self.k_scale,
                                    self.v_scale)
        self._address = ctypes.addressof(self._struct)

    def __setattr__(self, name, value):
        if "_address" in self.__dict__:
            raise AttributeError(f"a KVCache is fixed: make a new one to change {name}")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, dtype, device, k_scale: float = 1.0,
              v_scale: float = 1.0):
        """A new zero-filled cache with heads outermost within a page (a head's tokens contiguous)."""
        torch = _torch()
        k, v = (torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=torch.uint8 if dtype.itemsize == 1 else dtype,
                            device=device) for _ in range(2))
        if dtype.itemsize == 1:
            k, v = k.view(dtype), v.view(dtype)
        return cls(k.transpose(1, 2), v.transpose(1, 2), k_scale, v_scale)


def rope_table(rows: int, rot_dim: int, theta: float = 10000.0, device=None):
    """Rotation angles for positions 0..rows-1: fp32 [rows][rot_dim], the cosines of position * theta^(-2i/rot_dim)
    in the first half of a row and their sines in the second (computed in 64 bits)."""
    torch = _torch()
    half = rot_dim // 2
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * theta ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32).to(device)


def _int32(t, name: str, cache: KVCache, shape):
    if t.dtype is not cache._int32_type or t.get_device() != cache._index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on the cache's device")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _table(t, cache: KVCache):
    """Checks a block table; returns (pointer, columns, rows)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [sequences][columns]")
    return _int32(t, "block_table", cache, shape), shape[1], shape[0]


def _heads(t, name: str, shape, cache: KVCache, dtype):
    """Checks a [tokens][heads][head_dim] tensor (any token and head stride); returns (pointer, strides)."""
    if t.shape != shape:
        raise ValueError(f"{name} must be [tokens][heads][head_dim] = {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != cache._index:
        raise ValueError(f"{name} must live on the cache's device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: a head's values must be contiguous")
    return t.data_ptr(), ts, hs


def _queries(q, cache: KVCache, out):
    """Checks q and out (a new tensor if None): (shape, type id, out, q's pointer and strides, out's)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError(f"q must be [tokens][heads][head_dim of the cache], not {tuple(shape)}")
    dt = cache._acts.get(q.dtype)
    if dt is None:
        raise ValueError("activations must be float16 or bfloat16")
    if q.get_device() != cache._index:
        raise ValueError("q must live on the cache's device")
    ts, hs, one = q.stride()
    if one != 1:
        raise ValueError("q: a head's values must be contiguous")
    if out is None:
        out_hs = shape[2]
        out_ts = shape[1] * out_hs
        if hs == out_hs and ts == out_ts:
            out = cache._empty_like(q)   # keeps such strides
        else:
            out = cache._empty_like(q, memory_format=_torch().contiguous_format)
        oa = (out.data_ptr(), out_ts, out_hs)
    else:
        oa = _heads(out, "out", shape, cache, q.dtype)
    return shape, dt, out, (q.data_ptr(), ts, hs), oa


def _norm(w, name: str, cache: KVCache, dtype):
    if w is None:
        return 0
    if w.dtype is not dtype or w.get_device() != cache._index or w.shape != cache._norm_shape or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [head_dim] tensor of q's type")
    return w.data_ptr()


def qk_rope_append(q, k, v, positions, cache: KVCache, block_table, rope=None, q_norm=None, k_norm=None,
                   eps: float = 1e-6, token_seq=None, interleaved: bool = False, out=None):
    """Norms of queries and keys per head (q_norm, k_norm: [head_dim] weights or None), rotation by the rows of
    `rope` (``rope_table``) at `positions`, and the store of k and v into `cache`; returns the queries.

    q [tokens][q_heads][head_dim], k and v [tokens][kv_heads][head_dim], of any token and head strides (the parts of
    one fused product's output as they are); positions int32 [tokens] (negative: padding); block_table int32
    [sequences][columns]; token_seq int32 [tokens], or None when token t is sequence t's. `out` may be q."""
    shape, dt, out, qa, oa = _queries(q, cache, out)
    T, H, D = shape
    kv_shape, dtype = (T, cache.kv_heads, D), q.dtype
    rows, rot, rope_at = 1 << 24, 0, 0
    if rope is not None:
        if rope.dtype is not cache._float32_type or rope.dim() != 2 or rope.get_device() != cache._index or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 [positions][rot_dim] tensor")
        rows, rot = rope.shape
        rope_at = rope.data_ptr()
    table, cols, seqs = _table(block_table, cache)
    try:
        call = _append_call(
            *qa, *_heads(k, "k", kv_shape, cache, dtype), *_heads(v, "v", kv_shape, cache, dtype),
            _norm(q_norm, "q_norm", cache, dtype), _norm(k_norm, "k_norm", cache, dtype), rope_at, rows,
            _int32(positions, "positions", cache, (T,)),
            0 if token_seq is None else _int32(token_seq, "token_seq", cache, (T,)), table, cols, seqs, T,
            cache._address, *oa, cache._stream(cache._index), rot, 1 if interleaved else 0, H, dt, eps)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"qk_rope_append: {e}") from None
    status = lib().qgemm_qk_rope_append_call(call)
    if status:
        _check(status, "qgemm_qk_rope_append")
    return out


# Workspace sizes by shape and device: they depend on nothing else but the forced splits.
_ws_sizes = {}


def set_attn_splits(splits: int = 0):
    """Force the number of parts of the cache's length (0 = automatic); see include/qgemm.h."""
    _check(lib().qgemm_attn_set_splits(splits), "qgemm_attn_set_splits")
    _ws_sizes.clear()


def attn_decode_workspace_bytes(num_seqs: int, max_len: int, q_heads: int, kv_heads: int, head_dim: int,
                                window: int = 0, sinks: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().qgemm_attn_decode_workspace_bytes(num_seqs, max_len, q_heads, kv_heads, head_dim, window, sinks,
                                                   ctypes.byref(out)), "qgemm_attn_decode_workspace_bytes")
    return out.value


def attn_prefill_workspace_bytes(num_seqs: int, max_q: int, max_len: int, q_heads: int, kv_heads: int, head_dim: int,
                                 window: int = 0, sinks: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().qgemm_attn_prefill_workspace_bytes(num_seqs, max_q, max_len, q_heads, kv_heads, head_dim, window,
                                                    sinks, ctypes.byref(out)), "qgemm_attn_prefill_workspace_bytes")
    return out.value


def _workspace(workspace, cache, size_of, *shape):
    key = (size_of, cache._index, *shape)
    nbytes = _ws_sizes.get(key)
    if nbytes is None:
        if len(_ws_sizes) >= 4096:
            _ws_sizes.clear()
        nbytes = _ws_sizes[key] = size_of(*shape)
    if nbytes == 0:
        return 0, 0
    ws, wsb = (workspace or _default_ws).get(nbytes, cache.device)
    return ws.data_ptr(), wsb


def attn_decode(q, cache: KVCache, block_table, seq_lens, max_len: int, scale: float | None = None, window: int = 0,
                sinks: int = 0, out=None, workspace: Workspace | None = None):
    """Attention of one new token per sequence over its cached tokens (its own included): q [sequences][q_heads]
    [head_dim], block_table int32 [sequences][columns], seq_lens int32 [sequences], all at most max_len (a host number,
    so that the call reads nothing back; it sizes the grid and the workspace, so steps of a growing length do best with
    one bound for many of them, rounded up). window > 0 shows the last `window` tokens and the first `sinks`. scale
    defaults to head_dim ** -0.5. Returns q's shape and type."""
    shape, dt, out, qa, oa = _queries(q, cache, out)
    B, H, D = shape
    table, cols, seqs = _table(block_table, cache)
    if B != seqs:
        raise ValueError("q must have one row per sequence")
    lens = _int32(seq_lens, "seq_lens", cache, (B,))
    ws, wsb = _workspace(workspace, cache, attn_decode_workspace_bytes, B, max_len, H, cache.kv_heads, D, window,
                         sinks)
    try:
        call = _attn_call(*qa, cache._address, table, cols, 0, lens, B, B, 1, max_len, window, *oa, ws, wsb,
                          cache._stream(cache._index), H, dt, sinks, 1.0 / math.sqrt(D) if scale is None else scale)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"attn_decode: {e}") from None
    status = lib().qgemm_attn_decode_call(call)
    if status:
        _check(status, "qgemm_attn_decode")
    return out


def attn_prefill(q, cache: KVCache, block_table, q_start, seq_lens, max_q: int, max_len: int,
                 scale: float | None = None, window: int = 0, sinks: int = 0, out=None,
                 workspace: Workspace | None = None):
    """Causal attention of several new tokens per sequence: rows q_start[b]..q_start[b+1]-1 of q [tokens][q_heads]
    [head_dim] are the last tokens of sequence b, whose cache holds seq_lens[b] tokens with them. q_start int32
    [sequences + 1]; max_q and max_len bound the rows and lengths of every sequence (host numbers). Otherwise as
    attn_decode."""
    shape, dt, out, qa, oa = _queries(q, cache, out)
    T, H, D = shape
    table, cols, seqs = _table(block_table, cache)
    starts = _int32(q_start, "q_start", cache, (seqs + 1,))
    lens = _int32(seq_lens, "seq_lens", cache, (seqs,))
    ws, wsb = _workspace(workspace, cache, attn_prefill_workspace_bytes, seqs, max_q, max_len, H, cache.kv_heads, D,
                         window, sinks)
    try:
        call = _attn_call(*qa, cache._address, table, cols, starts, lens, seqs, T, max_q, max_len, window, *oa, ws, wsb,
                          cache._stream(cache._index), H, dt, sinks, 1.0 / math.sqrt(D) if scale is None else scale)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"attn_prefill: {e}") from None
    status = lib().qgemm_attn_prefill_call(call)
    if status:
        _check(status, "qgemm_attn_prefill")
    return out
