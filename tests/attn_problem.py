"""Paged-cache problems for the attention tests: NumPy inputs as bit patterns, device tensors, oracle outputs."""

import numpy as np
import torch

import bit_weight_quantized_qgemm_amd as qg
from oracle import attention as oa

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
NAN = {"f16": 0x7E00, "bf16": 0x7FC0, "fp8": 0x7F}


def to_torch(bits, fmt, dev):
    """Bit patterns (uint16 or uint8) as a device tensor of the format's type."""
    bits = np.ascontiguousarray(bits)
    t = torch.from_numpy(bits.view(np.int16 if bits.itemsize == 2 else np.uint8)).to(dev)
    return t.view(TORCH[fmt])


def to_bits(t):
    """A device tensor's bit patterns."""
    n = t.detach().contiguous()
    if n.element_size() == 1:
        return n.view(torch.uint8).cpu().numpy()
    return n.view(torch.int16).cpu().numpy().view(np.uint16)


class Paged:
    """A cache of `lens` tokens per sequence in shuffled pages, NaN in every place that holds no token, and a block
    table whose unused entries are out of range. layout: order of page, token and head in memory."""

    def __init__(self, rng, lens, kv_heads, dim, fmt, page, dev, layout="heads", scales=(1.0, 1.0), spare=2,
                 missing=()):
        self.lens, self.kv_heads, self.dim, self.fmt, self.page, self.scales = lens, kv_heads, dim, fmt, page, scales
        need = [-(-n // page) for n in lens]
        pool = sum(need) + spare
        order = rng.permutation(pool).astype(np.int32)
        cols = max(need + [0]) + 1
        self.table = np.full((len(lens), cols), -1, dtype=np.int32)
        self.table[:, -1] = np.iinfo(np.int32).max
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        dtype = np.uint8 if fmt == "fp8" else np.uint16
        # canonical [page][token][head][dim]
        self.bits = [np.full((pool, page, kv_heads, dim), NAN[fmt], dtype=dtype) for _ in range(2)]
        self.tokens = []   # per sequence: (k, v) as values
        for b, n in enumerate(lens):
            pair = []
            for i in range(2):
                x = rng.standard_normal((n, kv_heads, dim)) + (0.25 if i else 0.0)
                bits = oa.encode(x / scales[i], fmt)
                for j in range(n):
                    self.bits[i][self.table[b, j // page], j % page] = bits[j]
                pair.append(oa.decode(bits, fmt) * scales[i])
            self.tokens.append(pair)
        # pages that a sequence lost: their entries leave the range
        self.lost = np.zeros((len(lens), max(list(lens) + [1])), dtype=bool)
        for b, col, entry in missing:
            self.table[b, col] = entry if entry < 0 else pool + entry
            self.lost[b, col * page:(col + 1) * page] = True
        self.k, self.v = (self._place(x, layout, dev) for x in self.bits)
        self.cache = qg.KVCache(self.k, self.v, *scales)
        self.table_dev = torch.from_numpy(self.table).to(dev)
        self.lens_dev = torch.tensor(lens, dtype=torch.int32, device=dev)

    def _place(self, bits, layout, dev):
        pool, page, heads, dim = bits.shape
        fmt = self.fmt
        if layout == "heads":
            return to_torch(bits.transpose(0, 2, 1, 3), fmt, dev).transpose(1, 2)
        if layout == "tokens":
            return to_torch(bits, fmt, dev)
        # rows and heads padded, pages outermost, the whole at an offset
        assert layout == "padded"
        step = 16
        big = np.full((pool, heads, page + 1, dim + step), NAN[fmt], dtype=bits.dtype)
        big[:, :, :page, :dim] = bits.transpose(0, 2, 1, 3)
        return to_torch(big, fmt, dev)[:, :, :page, :dim].transpose(1, 2)

    def attend(self, b, q, pos, scale, window=0, sinks=0):
        """Oracle attention of one query (values [heads][dim]) of sequence b: (out, sum of weights |v|, score error,
        visible tokens)."""
        n = self.lens[b]
        see = oa.visible(pos, n, window, sinks) & ~self.lost[b, :n]
        group = q.shape[0] // self.kv_heads
        k, v = (np.repeat(x, group, axis=1) for x in self.tokens[b])
        return (*oa.attend(q, k, v, see, scale), int(see.sum()))


def check(got, refs, fmt, weight_roundoff, what):
    """got: values [rows][heads][dim]; refs: attend() of each row. Every output within its bound."""
    for r, (ref, mag, err, n) in enumerate(refs):
        bound = oa.attention_bound(ref, mag, err, n, fmt, weight_roundoff)
        if n == 0:
            assert not got[r].any(), (what, r)
            continue
        off = np.abs(got[r] - ref)
        assert np.all(off <= bound), (what, r, n, float((off / bound).max()))
