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

from . import DT_BF16, DT_F16, DT_FP8, Workspace, _check, _default_ws, _raw_stream, _torch, lib

__all__ = ["KVCache", "rope_table", "qk_rope_append", "attn_decode", "attn_prefill", "set_attn_splits",
           "attn_decode_workspace_bytes", "attn_prefill_workspace_bytes"]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


@functools.lru_cache(maxsize=None)
def _dtypes():
    torch = _torch()
    return {torch.float16: DT_F16, torch.bfloat16: DT_BF16, torch.float8_e4m3fn: DT_FP8}


class KVCache:
    """A paged key-value cache: k and v are [pages][page_size][kv_heads][head_dim] tensors (or views with the last
    dimension contiguous, the same strides for both), float16, bfloat16 or float8_e4m3fn; an e4m3 code stands for its
    value times k_scale (keys) or v_scale (values). Holds references, copies nothing."""

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
        self._index = k.device.index   # of the device whose current stream the calls use
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), self.num_pages, k.stride(0), k.stride(1), k.stride(2),
                                    self.page_size, self.kv_heads, self.head_dim, _dtypes()[k.dtype], self.k_scale,
                                    self.v_scale)
        self._ref = ctypes.byref(self._struct)

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


def _int32(t, name: str, device, shape):
    if t.dtype != _torch().int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on the cache's device")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")


def _table(t, device):
    if t.dim() != 2:
        raise ValueError("block_table must be [sequences][columns]")
    _int32(t, "block_table", device, t.shape)


def _heads(t, name: str, shape, cache: KVCache, dtype):
    """Checks a [tokens][heads][head_dim] tensor (any token and head stride); returns (pointer, strides)."""
    if t.shape != shape:
        raise ValueError(f"{name} must be [tokens][heads][head_dim] = {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != cache.device:
        raise ValueError(f"{name} must live on the cache's device")
    if t.dtype != dtype:
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
    dt = _dtypes().get(q.dtype)
    if dt is None or dt == DT_FP8:
        raise ValueError("activations must be float16 or bfloat16")
    qa = _heads(q, "q", shape, cache, q.dtype)
    if out is None:
        torch = _torch()
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    return shape, dt, out, qa, _heads(out, "out", shape, cache, q.dtype)


def qk_rope_append(q, k, v, positions, cache: KVCache, block_table, rope=None, q_norm=None, k_norm=None,
                   eps: float = 1e-6, token_seq=None, interleaved: bool = False, out=None):
    """Norms of queries and keys per head (q_norm, k_norm: [head_dim] weights or None), rotation by the rows of
    `rope` (``rope_table``) at `positions`, and the store of k and v into `cache`; returns the queries.

    q [tokens][q_heads][head_dim], k and v [tokens][kv_heads][head_dim], of any token and head strides (the parts of
    one fused product's output as they are); positions int32 [tokens] (negative: padding); block_table int32
    [sequences][columns]; token_seq int32 [tokens], or None when token t is sequence t's. `out` may be q."""
    torch = _torch()
    dev = cache.device
    shape, dt, out, qa, oa = _queries(q, cache, out)
    T, H, D = shape
    kv_shape = (T, cache.kv_heads, D)
    ka, va = _heads(k, "k", kv_shape, cache, q.dtype), _heads(v, "v", kv_shape, cache, q.dtype)
    _int32(positions, "positions", dev, (T,))
    _table(block_table, dev)
    if token_seq is not None:
        _int32(token_seq, "token_seq", dev, (T,))
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.dtype != q.dtype or w.device != dev or w.shape != (D,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous [head_dim] tensor of q's type")
    rows, rot = 1 << 24, 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 2 or rope.device != dev or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 [positions][rot_dim] tensor")
        rows, rot = rope.shape
    seqs, cols = block_table.shape
    _check(lib().qgemm_qk_rope_append(
        *qa, *ka, *va, None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
        eps, None if rope is None else rope.data_ptr(), rows, rot, 1 if interleaved else 0, positions.data_ptr(),
        None if token_seq is None else token_seq.data_ptr(), block_table.data_ptr(), cols, seqs, T, H, dt, cache._ref,
        *oa, _raw_stream(cache._index)), "qgemm_qk_rope_append")
    return out


def set_attn_splits(splits: int = 0):
    """Force the number of parts of the cache's length (0 = automatic); see include/qgemm.h."""
    _check(lib().qgemm_attn_set_splits(splits), "qgemm_attn_set_splits")


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


def _workspace(workspace, cache, nbytes):
    if nbytes == 0:
        return None, 0
    ws, wsb = (workspace or _default_ws).get(nbytes, cache.device)
    return ws.data_ptr(), wsb


def attn_decode(q, cache: KVCache, block_table, seq_lens, max_len: int, scale: float | None = None, window: int = 0,
                sinks: int = 0, out=None, workspace: Workspace | None = None):
    """Attention of one new token per sequence over its cached tokens (its own included): q [sequences][q_heads]
    [head_dim], block_table int32 [sequences][columns], seq_lens int32 [sequences], all at most max_len (a host number,
    so that the call reads nothing back). window > 0 shows the last `window` tokens and the first `sinks`. scale
    defaults to head_dim ** -0.5. Returns q's shape and type."""
    shape, dt, out, qa, oa = _queries(q, cache, out)
    B, H, D = shape
    dev = cache.device
    _table(block_table, dev)
    seqs, cols = block_table.shape
    if B != seqs:
        raise ValueError("q must have one row per sequence")
    _int32(seq_lens, "seq_lens", dev, (B,))
    ws, wsb = _workspace(workspace, cache,
                         attn_decode_workspace_bytes(B, max_len, H, cache.kv_heads, D, window, sinks))
    _check(lib().qgemm_attn_decode(
        *qa, cache._ref, block_table.data_ptr(), cols, seq_lens.data_ptr(), B, max_len, H, dt,
        1.0 / math.sqrt(D) if scale is None else scale, window, sinks, *oa, ws, wsb, _raw_stream(cache._index)),
        "qgemm_attn_decode")
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
    dev = cache.device
    _table(block_table, dev)
    seqs, cols = block_table.shape
    _int32(q_start, "q_start", dev, (seqs + 1,))
    _int32(seq_lens, "seq_lens", dev, (seqs,))
    ws, wsb = _workspace(workspace, cache,
                         attn_prefill_workspace_bytes(seqs, max_q, max_len, H, cache.kv_heads, D, window, sinks))
    _check(lib().qgemm_attn_prefill(
        *qa, cache._ref, block_table.data_ptr(), cols, q_start.data_ptr(), seq_lens.data_ptr(), seqs, T, max_q, max_len,
        H, dt, 1.0 / math.sqrt(D) if scale is None else scale, window, sinks, *oa, ws, wsb,
        _raw_stream(cache._index)), "qgemm_attn_prefill")
    return out
