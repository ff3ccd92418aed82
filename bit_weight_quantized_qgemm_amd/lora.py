"""Low-rank adapters of many requests beside a shared projection: the binding of the ``qgemm_lora*`` entry points of
``include/qgemm.h``.

As in the rest of the package: argument marshalling only, on the current HIP stream of the tensors' device, and no
fallback. Shapes, types and devices are checked here; strides, alignment, ranges and overlaps by the library, which
raises ``QgemmError``.
"""

from __future__ import annotations

import ctypes
import struct

from . import DT_BF16, DT_F16, Workspace, _check, _default_ws, _torch, lib

__all__ = ["LoraAdapters", "LoraBatch", "lora", "lora_workspace_bytes"]

MAX_SLICES = 8


class _AdaptersStruct(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("a_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("scales", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("widths", ctypes.c_int64 * MAX_SLICES),
                ("num_adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("slices", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


# The call's struct, packed into bytes: one argument through ctypes costs about as much as all of a struct's fields.
_lora_call = struct.Struct("@2PqPNPqPqqPNP").pack


class LoraAdapters:
    """The adapters of one projection, as a pool that requests choose from: a [adapters][rank][K] (or
    [adapters][slices][rank][K]) and b [adapters][N][rank], float16 or bfloat16, each adapter contiguous; scales float32
    [adapters] or None (1); ranks int32 [adapters] or None: the ranks of each adapter that count, up to a whole multiple
    of 8. widths: the columns of each slice of a fused projection (their sum is N), each of which has a first matrix of its
    own. Holds references, copies nothing, and is fixed: the calls take its addresses and strides as they were given here.
    What lies in the tensors may change: an adapter is replaced by writing over it."""

    def __init__(self, a, b, scales=None, ranks=None, widths=None):
        torch = _torch()
        if a.dtype not in (torch.float16, torch.bfloat16) or b.dtype != a.dtype:
            raise ValueError("a and b must both be float16 or bfloat16")
        if not a.is_cuda:
            raise ValueError("tensor must live on the GPU")
        if a.dim() == 3:
            a = a[:, None]
        if a.dim() != 4 or b.dim() != 3 or b.shape[0] != a.shape[0] or b.shape[2] != a.shape[2]:
            raise ValueError("a must be [adapters][slices][rank][K] and b [adapters][N][rank]")
        n, slices, rank, K = a.shape
        N = b.shape[1]
        widths = [N] if widths is None else [int(w) for w in widths]
        if len(widths) != slices or slices > MAX_SLICES or sum(widths) != N:
            raise ValueError(f"widths must be the columns of a's {slices} slices (at most {MAX_SLICES}), {N} in all")
        if n and (not a[0].is_contiguous() or not b[0].is_contiguous()):
            raise ValueError("each adapter's matrices must be contiguous")
        for t, name, dtype in ((scales, "scales", torch.float32), (ranks, "ranks", torch.int32)):
            if t is not None and (t.dtype != dtype or t.shape != (n,) or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of one value per adapter")
        for t in (b, scales, ranks):
            if t is not None and t.device != a.device:
                raise ValueError("all tensors must live on one device")
        self.a, self.b, self.scales, self.ranks = a, b, scales, ranks
        self.device, self.dtype, self._index = a.device, a.dtype, a.get_device()
        self.num_adapters, self.slices, self.rank, self.K, self.N = n, slices, rank, K, N
        self.widths = tuple(widths)
        # what every call looks up, at hand
        self._empty, self._stream, self._current = torch.empty, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self._struct = _AdaptersStruct(a.data_ptr(), b.data_ptr(), a.stride(0), b.stride(0),
                                       0 if scales is None else scales.data_ptr(), 0 if ranks is None else ranks.data_ptr(),
                                       K, N, (ctypes.c_int64 * MAX_SLICES)(*widths), n, rank, slices,
                                       DT_F16 if a.dtype == torch.float16 else DT_BF16)
        self._ws_bytes = {}   # by number of rows
        self._address = ctypes.addressof(self._struct)

    def __setattr__(self, name, value):
        if "_address" in self.__dict__:
            raise AttributeError(f"LoraAdapters are fixed: make new ones to change {name}")
        super().__setattr__(name, value)


class LoraBatch:
    """Which adapter each row of a batch uses: ids int32 [rows] on the GPU, outside 0..num_adapters-1 for none. Sorts the
    rows by adapter on the current stream, once for all projections of all layers that the batch goes through (their
    pools hold num_adapters adapters each). The ids are read here and not held; ``update`` sorts others of the same
    number, in the same memory, so that captured calls follow."""

    def __init__(self, ids, num_adapters: int):
        torch = _torch()
        if not ids.is_cuda:
            raise ValueError("tensor must live on the GPU")
        if ids.dim() != 1:
            raise ValueError("ids must be [rows]")
        self.rows, self.num_adapters, self.device, self._index = ids.shape[0], int(num_adapters), ids.device, ids.get_device()
        nbytes = ctypes.c_size_t(0)
        _check(lib().qgemm_lora_plan_bytes(self.rows, self.num_adapters, ctypes.byref(nbytes)), "qgemm_lora_plan_bytes")
        self.plan = torch.empty(nbytes.value, dtype=torch.uint8, device=ids.device)
        self._address, self._nbytes = self.plan.data_ptr(), nbytes.value
        self.update(ids)

    def update(self, ids):
        torch = _torch()
        if ids.dtype != torch.int32 or ids.shape != (self.rows,) or ids.device != self.device or not ids.is_contiguous():
            raise ValueError(f"ids must be a contiguous int32 tensor of {self.rows} rows on {self.device}")
        with torch.cuda.device(self._index):
            _check(lib().qgemm_lora_plan(ctypes.c_void_p(ids.data_ptr()), self.rows, self.num_adapters,
                                         ctypes.c_void_p(self._address), self._nbytes,
                                         ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(self._index))),
                   "qgemm_lora_plan")
        return self


def lora_workspace_bytes(rows: int, num_adapters: int, K: int, N: int, rank: int, slices: int = 1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().qgemm_lora_workspace_bytes(rows, num_adapters, K, N, rank, slices, ctypes.byref(out)),
           "qgemm_lora_workspace_bytes")
    return out.value


def _matrix(t, name: str, rows: int, cols: int, w: LoraAdapters):
    """Checks a [rows][cols] tensor of any row stride; returns (pointer, stride)."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [rows][columns] = {(rows, cols)}, not {tuple(t.shape)}")
    if t.dtype is not w.dtype or t.get_device() != w._index:
        raise ValueError(f"{name} must be {w.dtype} on the adapters' device")
    rs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    return t.data_ptr(), rs


def _launch(xa, ba, oa, rows: int, adapters: LoraAdapters, batch: LoraBatch, workspace):
    # a size depends on the device's compute units: looked up with it current
    nbytes = adapters._ws_bytes.get(rows)
    if nbytes is None:
        nbytes = adapters._ws_bytes[rows] = lora_workspace_bytes(rows, adapters.num_adapters, adapters.K, adapters.N,
                                                                 adapters.rank, adapters.slices)
    if nbytes == 0:
        return 0   # no rows
    ws, wsb = (workspace or _default_ws).get(nbytes, adapters.device)
    return lib().qgemm_lora(_lora_call(adapters._address, *xa, batch._address, batch._nbytes, *ba, *oa, rows, ws.data_ptr(),
                                       wsb, adapters._stream(adapters._index)))


def lora(x, adapters: LoraAdapters, batch: LoraBatch, base=None, out=None, workspace: Workspace | None = None):
    """base + scale * (x A^T) B^T with each row's own adapter: x [rows][K], base (or None) and out [rows][N] of any row
    strides. out may be base (the shared product's output, added to in place); rows without an adapter keep their base.
    Returns out, a new tensor if None."""
    if x.dim() != 2:
        raise ValueError("x must be [rows][K]")
    rows = x.shape[0]
    if batch.rows != rows or batch.num_adapters != adapters.num_adapters:
        raise ValueError(f"the batch is of {batch.rows} rows and {batch.num_adapters} adapters, the call of {rows} and "
                         f"{adapters.num_adapters}")
    if batch._index != adapters._index:
        raise ValueError("the batch must live on the adapters' device")
    xa = _matrix(x, "x", rows, adapters.K, adapters)
    ba = (0, 0) if base is None else _matrix(base, "base", rows, adapters.N, adapters)
    if out is None:
        out = adapters._empty((rows, adapters.N), dtype=adapters.dtype, device=adapters.device)
        oa = (out.data_ptr(), adapters.N)
    else:
        oa = _matrix(out, "out", rows, adapters.N, adapters)
    if adapters._current() == adapters._index:
        status = _launch(xa, ba, oa, rows, adapters, batch, workspace)
    else:
        with _torch().cuda.device(adapters._index):
            status = _launch(xa, ba, oa, rows, adapters, batch, workspace)
    if status:
        _check(status, "qgemm_lora")
    return out
